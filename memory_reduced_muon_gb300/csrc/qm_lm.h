// Shared by the operators on a model's activations (embedding.cu, mxfp8.cu,
// ffn.cu): 32-byte accesses, groups of 32 row elements, and what the host side
// asks of a device and of an argument.
#pragma once

#include <atomic>

#include "qm_elem.h"

namespace qm {
namespace lm {

// 32 bytes at once (one whole sector of a line), and 16.
__device__ __forceinline__ void store32b(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
               "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void load32b(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}

// How an array's rows may be accessed: 2 in 32-byte vectors, 1 in 16-byte ones, 0 by elements.
inline int vec_class(const void* p, int64_t ld, int es) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * es);
  return bits % 32 == 0 ? 2 : bits % 16 == 0 ? 1 : 0;
}

// 32 elements of a row (the first n of them where n < 32) as fp32, and back.
template <int DT>
__device__ __forceinline__ void load_row32(const void* p, int n, int vec, float (&v)[32]) {
  constexpr int es = elem_size(DT);
  if (n >= 32 && vec) {
    const unsigned char* b = static_cast<const unsigned char*>(p);
#pragma unroll
    for (int i = 0; i < es; ++i) {   // es x 32 bytes
      uint32_t w[8];
      if (vec == 2) {
        load32b(b + 32 * i, w);
      } else {
        const uint4 lo = *reinterpret_cast<const uint4*>(b + 32 * i), hi = *reinterpret_cast<const uint4*>(b + 32 * i + 16);
        w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w, w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (DT == QMUON_FP32) {
          v[8 * i + j] = __uint_as_float(w[j]);
        } else {
          const float2 f = unpack2<DT>(w[j]);
          v[16 * i + 2 * j] = f.x;
          v[16 * i + 2 * j + 1] = f.y;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = i < n ? load_elem<DT>(p, i) : 0.0f;
  }
}
// 32 elements of a 16-bit type as they lie in memory.
__device__ __forceinline__ void load_words32(const void* p, int n, int vec, uint32_t (&w)[16]) {
  if (n >= 32 && vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 q = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
    }
  } else {
    const uint16_t* e = static_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = (2 * i < n ? e[2 * i] : 0u) | ((2 * i + 1 < n ? (uint32_t)e[2 * i + 1] : 0u) << 16);
  }
}
template <int DT>
__device__ __forceinline__ void store_row32(void* p, int n, int vec, const float (&v)[32]) {
  constexpr int es = elem_size(DT);
  if (n >= 32 && vec) {
    unsigned char* b = static_cast<unsigned char*>(p);
#pragma unroll
    for (int i = 0; i < es; ++i) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (DT == QMUON_FP32) w[j] = __float_as_uint(v[8 * i + j]);
        else w[j] = pack2<DT>(v[16 * i + 2 * j], v[16 * i + 2 * j + 1]);
      }
      if (vec == 2) {
        store32b(b + 32 * i, w);
      } else {
        *reinterpret_cast<uint4*>(b + 32 * i) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(b + 32 * i + 16) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < n) store_elem<DT>(p, i, v[i]);
  }
}

// 32 codes of one MXFP8 scale, 16-byte aligned (vec: as above): E4M3 to the nearest of v times the power of two that the
// returned exponent byte stands for, and back, exactly in fp32.
__device__ __forceinline__ int encode_row32(uint8_t* p, int vec, const float (&v)[32]) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(v[i]));
  const int byte = e8m0_of_amax(amax);
  const float mult = pow2_from_e8m0(byte);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 a = mul2_rn(make_float2(v[4 * i], v[4 * i + 1]), mult), b = mul2_rn(make_float2(v[4 * i + 2], v[4 * i + 3]), mult);
    w[i] = cvt_e4m3x2(a.x, a.y) | (cvt_e4m3x2(b.x, b.y) << 16);
  }
  if (vec == 2) {
    store32b(p, w);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  }
  return byte;
}
// 2^(byte - 127): the subnormal 2^-127 for byte 0, NaN for 255.
__device__ __forceinline__ float scale_of_e8m0(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}
// Rounded to DT as a decoded checkpoint is: bf16 holds every product of a code
// and a scale down to its subnormals; in fp16 a finite value beyond its range
// is the largest that it has (the rounding up of a value that was within it).
template <int DT>
__device__ __forceinline__ float decoded(float v) {
  if constexpr (DT == QMUON_FP16) {
    if (fabsf(v) < INFINITY) v = fminf(fmaxf(v, -65504.0f), 65504.0f);
  }
  return v;
}

inline bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// SMs of the current device; 0 where the query fails.
inline int num_sms() {
  static std::atomic<int> cached[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < 64 && (n = cached[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

// mxfp8.cu: a carrier of rows x cols values (cols % 32 == 0) as rows of a type, ld elements apart; and the copy of
// rows of 16-bit elements to ones that start on 16 bytes.
cudaError_t launch_decode(const uint8_t* payload, const uint8_t* scale, void* x, int64_t rows, int64_t cols, int64_t ld, int dt,
                          cudaStream_t s);
cudaError_t launch_repack(const void* src, int64_t ld_src, void* dst, int64_t ld_dst, int64_t rows, int64_t cols, cudaStream_t s);

}  // namespace lm
}  // namespace qm
