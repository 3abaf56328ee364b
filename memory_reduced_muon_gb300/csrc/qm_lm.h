// Shared by the operators on a model's activations (embedding.cu, mxfp8.cu,
// ffn.cu): 32-byte accesses, groups of 32 row elements, and what the host side
// asks of a device and of an argument.
#pragma once

#include <atomic>

#include "qm_elem.h"

namespace qm {
namespace lm {

// A kernel's start: what follows it in the stream may be scheduled as soon as all of its CTAs have begun (it sets itself
// up meanwhile, and waits in turn); then what runs before it is complete.  See depends_wait.
__device__ __forceinline__ void depends_begin() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  depends_wait();
}

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

// W elements of a row (the first n of them where n < W) as fp32, and back:
// pieces of 64, 32 or 16 bytes, 16-byte aligned where vec is not 0.
template <int DT, int W>
__device__ __forceinline__ void load_row(const void* p, int n, int vec, float (&v)[W]) {
  constexpr int es = elem_size(DT), kBytes = W * es;
  static_assert(kBytes % 16 == 0, "whole vectors");
  if (n >= W && vec) {
    const unsigned char* b = static_cast<const unsigned char*>(p);
    uint32_t w[kBytes / 4];
    if (kBytes % 32 == 0 && vec == 2) {
#pragma unroll
      for (int i = 0; i < kBytes / 32; ++i) load32b(b + 32 * i, *reinterpret_cast<uint32_t(*)[8]>(w + 8 * i));
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 q = *reinterpret_cast<const uint4*>(b + 16 * i);
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
      }
    }
#pragma unroll
    for (int j = 0; j < kBytes / 4; ++j) {
      if constexpr (DT == QMUON_FP32) {
        v[j] = __uint_as_float(w[j]);
      } else {
        const float2 f = unpack2<DT>(w[j]);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = i < n ? load_elem<DT>(p, i) : 0.0f;
  }
}
template <int DT, int W>
__device__ __forceinline__ void store_row(void* p, int n, int vec, const float (&v)[W]) {
  constexpr int es = elem_size(DT), kBytes = W * es;
  static_assert(kBytes % 16 == 0, "whole vectors");
  if (n >= W && vec) {
    unsigned char* b = static_cast<unsigned char*>(p);
    uint32_t w[kBytes / 4];
#pragma unroll
    for (int j = 0; j < kBytes / 4; ++j) {
      if constexpr (DT == QMUON_FP32) w[j] = __float_as_uint(v[j]);
      else w[j] = pack2<DT>(v[2 * j], v[2 * j + 1]);
    }
    if (kBytes % 32 == 0 && vec == 2) {
#pragma unroll
      for (int i = 0; i < kBytes / 32; ++i) store32b(b + 32 * i, *reinterpret_cast<uint32_t(*)[8]>(w + 8 * i));
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        *reinterpret_cast<uint4*>(b + 16 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (i < n) store_elem<DT>(p, i, v[i]);
  }
}

// The same for every lane of a converged warp (p, n: the lane's own, n = 0 for
// none; vec alike in all of them).  Rows that cannot be accessed in vectors go
// through `stage`, 32 W fp32 of the warp's own, so that neighbouring lanes
// access neighbouring elements: 32 lanes that each write a row of their own
// touch 32 sectors with every 2-byte store.
template <int W>
__device__ __forceinline__ int stage_at(int row, int col) {
  return row * W + (col ^ (row & (W - 1)));   // column k of all rows in different banks (in pairs for W < 32)
}
// (Functions of their own: in line, their registers would cost the kernels that reach them only with unaligned rows.)
template <int DT, int W>
__device__ __noinline__ void fill_stage(const void* p, int n, float* stage) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int j0 = 0; j0 < W; j0 += 8) {   // eight at a time: shuffles, accesses of either memory
    float e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = ((j0 + j) * 32 + lane) / W, col = ((j0 + j) * 32 + lane) % W;
      const int m = __shfl_sync(0xffffffffu, n, row);
      const void* q = reinterpret_cast<const void*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(p), row));
      e[j] = 0.0f;
      if (col < m) e[j] = load_elem<DT>(q, col);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) stage[stage_at<W>(((j0 + j) * 32 + lane) / W, ((j0 + j) * 32 + lane) % W)] = e[j];
  }
  __syncwarp();
}
template <int DT, int W>
__device__ __noinline__ void drain_stage(void* p, int n, const float* stage) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int j0 = 0; j0 < W; j0 += 8) {
    float e[8];
    int m[8];
    uintptr_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = ((j0 + j) * 32 + lane) / W, col = ((j0 + j) * 32 + lane) % W;
      e[j] = stage[stage_at<W>(row, col)];
      m[j] = __shfl_sync(0xffffffffu, n, row) - col;
      q[j] = __shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(p), row) + col * elem_size(DT);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (m[j] > 0) store_elem<DT>(reinterpret_cast<void*>(q[j]), 0, e[j]);
  }
  __syncwarp();
}
template <int DT, int W>
__device__ __forceinline__ void load_rows(const void* p, int n, int vec, float (&v)[W], float* stage) {
  if (vec) {
    load_row<DT, W>(p, n, vec, v);
    return;
  }
  fill_stage<DT, W>(p, n, stage);
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < W; ++k) v[k] = stage[stage_at<W>(lane, k)];
}
template <int DT, int W>
__device__ __forceinline__ void store_rows(void* p, int n, int vec, const float (&v)[W], float* stage) {
  if (vec) {
    store_row<DT, W>(p, n, vec, v);
    return;
  }
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < W; ++k) stage[stage_at<W>(lane, k)] = v[k];
  drain_stage<DT, W>(p, n, stage);
}

// W codes (16 or 32) of an MXFP8 scale of 32, 16-byte aligned (vec: as above): E4M3 to the nearest of v times the power of
// two that the returned exponent byte stands for.  W = 16: lanes 2 i and 2 i + 1 share the scale, and every lane of the
// warp calls this; `valid`: whether the lane has codes to write.
template <int W>
__device__ __forceinline__ int encode_row(uint8_t* p, bool valid, int vec, const float (&v)[W]) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) amax = fmaxf(amax, fabsf(v[i]));
  if constexpr (W == 16) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  const int byte = e8m0_of_amax(amax);
  const float mult = pow2_from_e8m0(byte);
  uint32_t w[W / 4];
#pragma unroll
  for (int i = 0; i < W / 4; ++i) {
    const float2 a = mul2_rn(make_float2(v[4 * i], v[4 * i + 1]), mult), b = mul2_rn(make_float2(v[4 * i + 2], v[4 * i + 3]), mult);
    w[i] = cvt_e4m3x2(a.x, a.y) | (cvt_e4m3x2(b.x, b.y) << 16);
  }
  if (valid) {
    if constexpr (W == 32) {
      if (vec == 2) {
        store32b(p, w);
        return byte;
      }
    }
#pragma unroll
    for (int i = 0; i < W / 16; ++i) *reinterpret_cast<uint4*>(p + 16 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  return byte;
}
// W codes under one scale as fp32, exactly.
template <int W>
__device__ __forceinline__ void decode_row(const uint8_t* p, int vec, float scale, float (&v)[W]) {
  uint32_t w[W / 4];
  bool done = false;
  if constexpr (W == 32) {
    if (vec == 2) {
      load32b(p, w);
      done = true;
    }
  }
  if (!done) {
#pragma unroll
    for (int i = 0; i < W / 16; ++i) {
      const uint4 q = *reinterpret_cast<const uint4*>(p + 16 * i);
      w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
    }
  }
#pragma unroll
  for (int i = 0; i < W / 4; ++i) {
    const float2 a = mul2_rn(e4m3x2_to(w[i] & 0xFFFFu), scale), c = mul2_rn(e4m3x2_to(w[i] >> 16), scale);
    v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = c.x, v[4 * i + 3] = c.y;
  }
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

// mxfp8.cu: a carrier of rows x cols values (cols % 32 == 0) as rows of a type, ld elements apart; and the copies of
// up to three matrices of 16-bit elements to rows that start on 16 bytes.
cudaError_t launch_decode(const uint8_t* payload, const uint8_t* scale, void* x, int64_t rows, int64_t cols, int64_t ld, int dt,
                          cudaStream_t s);
struct Repack {
  const uint16_t* src;
  uint16_t* dst;
  int64_t ld_src, ld_dst, rows, cols;
};
cudaError_t launch_repack(const Repack* jobs, int n, cudaStream_t s);

}  // namespace lm
}  // namespace qm
