// Element types of the training operators (adamw.cu, rmsnorm.cu): widening
// and rounding between the stored types and fp32, 16-byte vectors, E4M3 codes
// and the Philox generator.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qm_internal.h"

namespace qm {

__host__ __device__ constexpr int elem_size(int dt) { return dt == QMUON_FP32 ? 4 : 2; }

// One stored element of type DT as fp32, and back (nearest even).
template <int DT>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (DT == QMUON_FP32) return static_cast<const float*>(p)[i];
  if constexpr (DT == QMUON_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float v) {
  if constexpr (DT == QMUON_FP32) static_cast<float*>(p)[i] = v;
  if constexpr (DT == QMUON_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  if constexpr (DT == QMUON_FP16) static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// A 32-bit word of two 16-bit elements.
template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (DT == QMUON_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == QMUON_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A 16-byte vector of DT as fp32 values: 8 of a 16-bit type, 4 of fp32.
template <int DT>
struct Vec16 {
  static constexpr int kElems = 16 / elem_size(DT);
  __device__ __forceinline__ static void unpack(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == QMUON_FP32) {
        f[i] = __uint_as_float(w[i]);
      } else {
        const float2 t = unpack2<DT>(w[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
      }
    }
  }
  __device__ __forceinline__ static uint4 pack(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == QMUON_FP32) w[i] = __float_as_uint(f[i]);
      else w[i] = pack2<DT>(f[2 * i], f[2 * i + 1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Two E4M3 codes (the low one first) from fp32, nearest even, |x| > 448
// saturating, NaN to 0x7F; and back, exactly.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return (uint32_t)r;
}
__device__ __forceinline__ float2 e4m3x2_to(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// E8M0 exponent byte of a block of 32: 127 + e with e the smallest integer
// such that amax <= 448 2^e, clamped to [0, 254]; 127 for amax == 0, 254 for
// an infinite one.  With amax = f 2^E, f in [1, 2), e = E - 8 + [f > 1.75].
__device__ __forceinline__ int e8m0_byte(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int ef = (int)(b >> 23);
  const int byte = ef - 8 + (((b & 0x7FFFFFu) > 0x600000u) ? 1 : 0);
  return b == 0u ? 127 : (ef == 0xFF ? 254 : min(max(byte, 0), 254));
}
// 2^(127 - byte); byte 254 gives the subnormal 2^-127.
__device__ __forceinline__ float e8m0_inverse(int byte) {
  return __uint_as_float(byte < 254 ? (uint32_t)(254 - byte) << 23 : 0x00400000u);
}

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC'11).
__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint32_t hi0 = __umulhi(0xD2511F53u, c.x), lo0 = 0xD2511F53u * c.x;
    const uint32_t hi1 = __umulhi(0xCD9E8D57u, c.z), lo1 = 0xCD9E8D57u * c.z;
    c = make_uint4(hi1 ^ c.y ^ k0, lo1, hi0 ^ c.w ^ k1, lo0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

}  // namespace qm
