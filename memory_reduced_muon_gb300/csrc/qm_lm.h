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

inline bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

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

// The W columns of a row that a thread takes.  Side by side from column c, n of them there: rows on 16 bytes, in vectors
// (vec not 0).  ANY: rows that start anywhere; columns c, c + 32, ..., n of them there, lane l of the warp's having c + l:
// neighbouring lanes access neighbouring elements, in which a warp's 2-byte accesses touch 3 sectors (32 if each lane had
// columns of its own side by side).
template <int W, bool ANY>
struct Columns {
  int64_t c;
  int n;
  template <int DT>
  __device__ __forceinline__ void load(const void* row, int vec, float (&v)[W]) const {
    if constexpr (ANY) {
#pragma unroll
      for (int k = 0; k < W; ++k) v[k] = k < n ? load_elem<DT>(row, c + 32 * k) : 0.0f;
    } else {
      load_row<DT, W>(static_cast<const unsigned char*>(row) + c * elem_size(DT), n, vec, v);
    }
  }
  template <int DT>
  __device__ __forceinline__ void store(void* row, int vec, const float (&v)[W]) const {
    if constexpr (ANY) {
#pragma unroll
      for (int k = 0; k < W; ++k)
        if (k < n) store_elem<DT>(row, c + 32 * k, v[k]);
    } else {
      store_row<DT, W>(static_cast<unsigned char*>(row) + c * elem_size(DT), n, vec, v);
    }
  }
};
__device__ __forceinline__ int valid_columns(int64_t left, int most) { return left >= most ? most : left > 0 ? (int)left : 0; }
// Thread i's columns, and its row, of rows x cols dealt out to threads (ANY: to warps of a row); no columns behind the last.
template <int W, bool ANY>
__device__ __forceinline__ Columns<W, ANY> deal_columns(int64_t i, int64_t rows, int64_t cols, int64_t* row) {
  Columns<W, ANY> t{0, 0};
  const int64_t per = ANY ? (cols + 32 * W - 1) / (32 * W) * 32 : (cols + W - 1) / W;
  *row = 0;
  if (i < rows * per) {
    *row = i / per;
    const int64_t j = i - *row * per;
    if constexpr (ANY) {
      t.c = (j >> 5) * (32 * W) + (j & 31);
      t.n = valid_columns((cols - t.c + 31) >> 5, W);
    } else {
      t.c = j * W;
      t.n = valid_columns(cols - t.c, W);
    }
  }
  return t;
}
inline int64_t threads_of(int64_t rows, int64_t cols, int w, bool any) {
  return rows * (any ? ceil_div(cols, 32 * w) * 32 : ceil_div(cols, w));
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
// The codes of a row's columns, and their exponents (`row`: the row's codes, `scales`: its exponents, valid where there are
// columns).  Every lane of the warp calls them.
template <int W, bool ANY>
__device__ __forceinline__ void encode_columns(const Columns<W, ANY>& t, uint8_t* row, uint8_t* scales, int vec, const float (&v)[W]) {
  if constexpr (ANY) {
#pragma unroll
    for (int k = 0; k < W; ++k) {   // a scale's 32 columns are the warp's lanes'
      const float a = k < t.n ? fmaxf(fabsf(v[k]), 0.0f) : 0.0f;   // not negative, no NaN: ordered as integers
      const int byte = e8m0_of_amax(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a))));
      if (k >= t.n) continue;
      row[t.c + 32 * k] = (uint8_t)cvt_e4m3x2(__fmul_rn(v[k], pow2_from_e8m0(byte)), 0.0f);
      if ((t.c & 31) == 0) scales[(t.c >> 5) + k] = (uint8_t)byte;
    }
  } else {
    const int byte = encode_row<W>(row + t.c, t.n > 0, vec, v);
    if (t.n > 0 && (t.c & 31) == 0) scales[t.c >> 5] = (uint8_t)byte;
  }
}
// 2^(byte - 127): the subnormal 2^-127 for byte 0, NaN for 255.
__device__ __forceinline__ float scale_of_e8m0(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}
template <int W, bool ANY>
__device__ __forceinline__ void decode_columns(const Columns<W, ANY>& t, const uint8_t* row, const uint8_t* scales, int vec, float (&v)[W]) {
  if constexpr (ANY) {
#pragma unroll
    for (int k = 0; k < W; ++k)
      v[k] = k < t.n ? __fmul_rn(e4m3x2_to(row[t.c + 32 * k]).x, scale_of_e8m0(scales[(t.c >> 5) + k])) : 0.0f;
  } else {
    if (t.n > 0) decode_row<W>(row + t.c, vec, scale_of_e8m0(scales[t.c >> 5]), v);
  }
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
