// Device helpers shared by update.cu, adamw.cu, rmsnorm.cu and, through qm_lm.h,
// embedding.cu, mxfp8.cu and ffn.cu: widening and
// rounding between the stored types and fp32, 16-byte vectors, packed fp32
// pairs, E4M3 codes and E8M0 scales, asynchronous copies, dependent launches,
// and the Philox generator under round keys made on the host.
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

// A 16-byte vector of DT as fp32 pairs: 8 values of a 16-bit type, 4 of fp32.
template <int DT>
struct Vec16 {
  static constexpr int kElems = 16 / elem_size(DT);
  static constexpr int kPairs = kElems / 2;
  __device__ __forceinline__ static void unpack(const uint4& v, float2* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (DT == QMUON_FP32) {
      f[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
      f[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = unpack2<DT>(w[i]);
    }
  }
  __device__ __forceinline__ static uint4 pack(const float2* f) {
    if constexpr (DT == QMUON_FP32)
      return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    else
      return make_uint4(pack2<DT>(f[0].x, f[0].y), pack2<DT>(f[1].x, f[1].y), pack2<DT>(f[2].x, f[2].y),
                        pack2<DT>(f[3].x, f[3].y));
  }
};

// Packed fp32 pairs (one instruction for two lanes of arithmetic), each
// component rounded to nearest exactly as the scalar __fmul_rn / __fsub_rn.
// ptxas fuses a packed multiply whose only use is a packed add into a packed
// FMA (one rounding instead of two), so a product that feeds an addition is
// always added with the scalar __fadd_rn: those chains were checked bit for
// bit against the scalar ones on the GPU (sub -> mul, mul -> scalar add,
// mul -> max -> add, mul -> E4M3 conversion).
__device__ __forceinline__ float2 mul2_rn(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 pa, pb, pd;\n\tmov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
      "mul.rn.f32x2 pd, pa, pb;\n\tmov.b64 {%0, %1}, pd;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 sub2_rn(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 pa, pb, pd;\n\tmov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
      "sub.rn.f32x2 pd, pa, pb;\n\tmov.b64 {%0, %1}, pd;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ float2 mul2_rn(float2 a, float b) { return mul2_rn(a, make_float2(b, b)); }
// Rounded towards zero.
__device__ __forceinline__ float2 mul2_rz(float2 a, float b) {
  float2 r;
  asm("{\n\t.reg .b64 pa, pb, pd;\n\tmov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %4};\n\t"
      "mul.rz.f32x2 pd, pa, pb;\n\tmov.b64 {%0, %1}, pd;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 pa, pb, pd;\n\tmov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
      "add.rn.f32x2 pd, pa, pb;\n\tmov.b64 {%0, %1}, pd;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 pa, pb, pc, pd;\n\tmov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\tmov.b64 pc, {%6, %7};\n\t"
      "fma.rn.f32x2 pd, pa, pb, pc;\n\tmov.b64 {%0, %1}, pd;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// Asynchronous copies of the calling thread into shared memory.
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Every kernel of these operators is launched as a programmatic dependent of
// what runs before it in its stream: it may start while that drains (and lets
// its own successor do so), and touches nothing that others write before
// depends_wait() has returned, which is once that has completed.  Every thread
// calls it, so that a kernel never completes before its predecessor.  Loads of
// what others write are plain ones: a load that may use the read-only path
// (__ldg) is not held back by the wait.
__device__ __forceinline__ void depends_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <class... Params, class... Args>
inline cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

// Two E4M3 codes (the low one first) from fp32, nearest even, |x| > 448
// saturating, NaN to 0x7F; and back, exactly.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return (uint32_t)r;
}

__device__ __forceinline__ float2 e4m3x2_to(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// E8M0 exponent byte of a 32-element block: 127 + e with e the smallest
// integer such that amax <= 448 * 2^e (448 = 1.75 * 2^8 is the largest E4M3
// value), clamped to [0, 254]; 127 for amax == 0, 254 for amax == inf.
// With amax = f * 2^E (f in [1, 2), biased exponent field ef = E + 127),
// e = E - 8 + [f > 1.75], so the byte is ef - 8 + [mantissa > 0.75].  A
// subnormal amax (ef = 0, below 2^-126) and any amax below 2^-119 give a
// negative byte and clamp to 0, so no subnormal case is needed: the byte is
// a few integer operations and selects, without branches.
__device__ __forceinline__ int e8m0_of_amax(float amax) {
  const uint32_t b = __float_as_uint(amax);   // amax >= 0: the sign bit is clear
  const int ef = (int)(b >> 23);
  const int byte = ef - 8 + (((b & 0x7FFFFFu) > 0x600000u) ? 1 : 0);
  const int clamped = byte < 0 ? 0 : (byte > 254 ? 254 : byte);
  return b == 0u ? 127 : (ef == 0xFF ? 254 : clamped);
}

// 2^(127 - byte) as an fp32 (byte in [0, 254]: exponent in [-127, 127]); the
// one subnormal power, 2^-127 (byte 254), is the pattern 0x00400000.
__device__ __forceinline__ float pow2_from_e8m0(int byte) {
  return __uint_as_float(byte < 254 ? (uint32_t)(254 - byte) << 23 : 0x00400000u);
}

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC'11) under the round keys of a seed, made on the host.
struct PhiloxKeys {
  uint32_t k[10][2];
  void set(uint64_t seed) {
    for (int r = 0; r < 10; ++r) {
      k[r][0] = (uint32_t)seed + (uint32_t)r * 0x9E3779B9u;
      k[r][1] = (uint32_t)(seed >> 32) + (uint32_t)r * 0xBB67AE85u;
    }
  }
};
__device__ __forceinline__ uint4 philox(uint4 c, const PhiloxKeys& key) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * c.x, p1 = (uint64_t)0xCD9E8D57u * c.z;
    c = make_uint4((uint32_t)(p1 >> 32) ^ c.y ^ key.k[r][0], (uint32_t)p1, (uint32_t)(p0 >> 32) ^ c.w ^ key.k[r][1],
                   (uint32_t)p0);
  }
  return c;
}

}  // namespace qm
