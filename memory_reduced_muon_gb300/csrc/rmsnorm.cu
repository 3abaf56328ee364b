// RMS norm with the residual's addition, forward (same-type or MXFP8 output)
// and backward.
//
//   h = x + residual          y = h / sqrt(mean(h^2) + eps) * gain
//   a = dy * gain, n = h inv: dx = inv (a - n mean(a n)) + dsum
//                             dgain = sum over rows of dy n
//
// A row is held in registers by T threads (a power of two up to a warp, or
// whole warps), V vectors of 16 bytes each, from its loads to its stores, so
// that every array crosses HBM once.  Rows that start off a 16-byte boundary
// are moved element by element; rows longer than the registers of 1024
// threads hold are read twice.
#include <algorithm>
#include <cmath>

#include "qm_elem.h"

namespace qm {
namespace {

constexpr int kMaxT = 1024;

struct FwdArgs {
  const void* x;
  const void* residual;   // or null
  const float* gain;
  void* sum;              // or null
  void* y;                // or null
  uint8_t* payload;       // MXFP8 output, or null
  uint8_t* scale;
  int64_t rows, ld_x, ld_residual, ld_sum, ld_y;
  int32_t cols;
  float eps, inv_cols;
};

struct BwdArgs {
  const void* dy;
  const void* h;
  const void* dsum;       // or null
  const float* gain;
  void* dx;
  float* partial;         // [grid][cols]
  int64_t rows, ld_dy, ld_h, ld_dsum, ld_dx;
  int32_t cols;
  float eps, inv_cols;
};

// VEC consecutive elements (one 16-byte vector, or one element) at index i.
template <int DT, int VEC>
__device__ __forceinline__ void load_vec(const void* row, int i, float* f) {
  if constexpr (VEC == 1) f[0] = load_elem<DT>(row, i);
  else Vec16<DT>::unpack(reinterpret_cast<const uint4*>(row)[i], f);
}
template <int DT, int VEC>
__device__ __forceinline__ void store_vec(void* row, int i, const float* f) {
  if constexpr (VEC == 1) store_elem<DT>(row, i, f[0]);
  else reinterpret_cast<uint4*>(row)[i] = Vec16<DT>::pack(f);
}
template <int DT>
__device__ __forceinline__ const void* row_of(const void* base, int64_t row, int64_t ld) {
  return static_cast<const unsigned char*>(base) + row * ld * elem_size(DT);
}
template <int DT>
__device__ __forceinline__ void* row_of(void* base, int64_t row, int64_t ld) {
  return static_cast<unsigned char*>(base) + row * ld * elem_size(DT);
}
template <int VEC>
__device__ __forceinline__ void load_gain(const float* gain, int i, float* f) {
  if constexpr (VEC == 1) {
    f[0] = __ldg(gain + i);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; j += 4) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(gain + (int64_t)i * VEC + j));
      f[j] = t.x, f[j + 1] = t.y, f[j + 2] = t.z, f[j + 3] = t.w;
    }
  }
}

// Sum of v over the T threads of a row (the same in all of them).  T > 32:
// `part` is one float per warp; the caller alternates two of them, so that one
// barrier per sum is enough.
__device__ __forceinline__ float row_sum(float v, int T, float* part) {
  for (int o = min(T, 32) >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (T <= 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = T >> 5;
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < nw ? part[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The MXFP8 codes of VEC values held by a thread whose neighbours hold the
// rest of the 32-element block; every thread of the warp calls it.
template <int DT, int VEC>
__device__ __forceinline__ void store_mxfp8(const float* y, bool valid, int64_t e, uint8_t* payload, uint8_t* scale) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < VEC; ++j) amax = fmaxf(amax, valid ? fabsf(y[j]) : 0.0f);
#pragma unroll
  for (int o = 16 / VEC; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int byte = e8m0_byte(amax);
  const float mult = e8m0_inverse(byte);
  if (!valid) return;
  if constexpr (VEC == 1) {
    payload[e] = (uint8_t)e4m3x2_of(__fmul_rn(y[0], mult), 0.0f);
  } else {
    uint32_t w[VEC / 4];
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j)
      w[j] = e4m3x2_of(__fmul_rn(y[4 * j], mult), __fmul_rn(y[4 * j + 1], mult)) |
             (e4m3x2_of(__fmul_rn(y[4 * j + 2], mult), __fmul_rn(y[4 * j + 3], mult)) << 16);
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(payload + e) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(payload + e) = w[0];
  }
  if ((e & 31) == 0) scale[e >> 5] = (uint8_t)byte;
}

// blockDim = (T, rows per CTA); T > 32 has one row per CTA.
template <int DT, int VEC, int V, bool MX>
__global__ void __launch_bounds__(kMaxT) rmsnorm_fwd_kernel(const __grid_constant__ FwdArgs A) {
  __shared__ float part[2][32];
  const int T = blockDim.x, t = threadIdx.x;
  const int nv = A.cols / VEC;
  int flip = 0;
  // rows per pass are the same for the whole grid, so every thread of a warp leaves the loop together
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < A.rows; r0 += (int64_t)gridDim.x * blockDim.y, flip ^= 1) {
    const int64_t row = r0 + threadIdx.y;
    const bool live = row < A.rows;
    const int n = live ? nv : 0;
    const void* x = row_of<DT>(A.x, row, A.ld_x);
    float h[V][VEC];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = i * T + t;
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[i][j] = 0.0f;
      if (k < n) load_vec<DT, VEC>(x, k, h[i]);
    }
    if (A.residual) {
      const void* res = row_of<DT>(A.residual, row, A.ld_residual);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int k = i * T + t;
        if (k < n) {
          float f[VEC];
          load_vec<DT, VEC>(res, k, f);
#pragma unroll
          for (int j = 0; j < VEC; ++j) h[i][j] += f[j];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    if (A.sum) {
      void* sum = row_of<DT>(A.sum, row, A.ld_sum);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i * T + t < n) store_vec<DT, VEC>(sum, i * T + t, h[i]);
    }
    ss = row_sum(ss, T, part[flip]);
    const float inv = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(ss, A.inv_cols, A.eps)));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = i * T + t;
      float g[VEC];
      if (k < n) {
        load_gain<VEC>(A.gain, k, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[i][j] = h[i][j] * inv * g[j];
        if (A.y) store_vec<DT, VEC>(row_of<DT>(A.y, row, A.ld_y), k, h[i]);
      }
      if constexpr (MX) store_mxfp8<DT, VEC>(h[i], k < n, row * A.cols + (int64_t)k * VEC, A.payload, A.scale);
    }
  }
}

// Rows that do not fit the registers of a CTA: read for the sum, and again for the output.
template <int DT, int VEC, bool MX>
__global__ void __launch_bounds__(kMaxT) rmsnorm_fwd_long_kernel(const __grid_constant__ FwdArgs A) {
  __shared__ float part[2][32];
  const int T = blockDim.x, t = threadIdx.x;
  const int nv = A.cols / VEC;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x, flip ^= 1) {
    const void* x = row_of<DT>(A.x, row, A.ld_x);
    const void* res = row_of<DT>(A.residual, row, A.ld_residual);
    auto load = [&](int k, float* h) {
      load_vec<DT, VEC>(x, k, h);
      if (A.residual) {
        float f[VEC];
        load_vec<DT, VEC>(res, k, f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[j] += f[j];
      }
    };
    float ss = 0.0f;
    for (int k = t; k < nv; k += T) {
      float h[VEC];
      load(k, h);
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss = fmaf(h[j], h[j], ss);
    }
    ss = row_sum(ss, T, part[flip]);
    const float inv = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(ss, A.inv_cols, A.eps)));
    for (int k0 = 0; k0 < nv; k0 += T) {   // the same number of passes in every thread
      const int k = k0 + t;
      float h[VEC] = {}, g[VEC];
      if (k < nv) {
        load(k, h);
        if (A.sum) store_vec<DT, VEC>(row_of<DT>(A.sum, row, A.ld_sum), k, h);
        load_gain<VEC>(A.gain, k, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) h[j] = h[j] * inv * g[j];
        if (A.y) store_vec<DT, VEC>(row_of<DT>(A.y, row, A.ld_y), k, h);
      }
      if constexpr (MX) store_mxfp8<DT, VEC>(h, k < nv, row * A.cols + (int64_t)k * VEC, A.payload, A.scale);
    }
  }
}

// Two sums over the T threads of a row.
__device__ __forceinline__ float2 row_sum2(float2 v, int T, float2* part) {
  for (int o = min(T, 32) >> 1; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if (T <= 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = T >> 5;
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < nw ? part[lane] : make_float2(0.0f, 0.0f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  return v;
}

// The backward pass: a CTA's threads keep the gain of their columns and its
// gradient over all rows of the CTA, which then leaves as one row of
// `partial`; dgain_kernel adds those rows in order.
template <int DT, int VEC, int V>
__global__ void __launch_bounds__(V * VEC >= 16 ? 512 : kMaxT) rmsnorm_bwd_kernel(const __grid_constant__ BwdArgs A) {
  __shared__ float2 part[2][32];
  extern __shared__ float s_gain[];   // T <= 32: [rows per CTA][cols]
  const int T = blockDim.x, t = threadIdx.x;
  const int nv = A.cols / VEC;
  float acc[V][VEC], gain[V][VEC];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[i][j] = gain[i][j] = 0.0f;
    if (i * T + t < nv) load_gain<VEC>(A.gain, i * T + t, gain[i]);
  }
  int flip = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < A.rows; r0 += (int64_t)gridDim.x * blockDim.y, flip ^= 1) {
    const int64_t row = r0 + threadIdx.y;
    const int n = row < A.rows ? nv : 0;
    const void* hp = row_of<DT>(A.h, row, A.ld_h);
    const void* dp = row_of<DT>(A.dy, row, A.ld_dy);
    float h[V][VEC], d[V][VEC];
    float2 s = make_float2(0.0f, 0.0f);   // sum h^2, sum a h
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[i][j] = d[i][j] = 0.0f;
      if (i * T + t < n) {
        load_vec<DT, VEC>(hp, i * T + t, h[i]);
        load_vec<DT, VEC>(dp, i * T + t, d[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        s.x = fmaf(h[i][j], h[i][j], s.x);
        s.y = fmaf(d[i][j] * gain[i][j], h[i][j], s.y);
      }
    s = row_sum2(s, T, part[flip]);
    const float inv = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(s.x, A.inv_cols, A.eps)));
    const float c = s.y * A.inv_cols * inv * inv;   // mean(a h) inv^2
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = i * T + t;
      if (k < n) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          o[j] = inv * (d[i][j] * gain[i][j] - h[i][j] * c);
          acc[i][j] = fmaf(d[i][j], h[i][j] * inv, acc[i][j]);
        }
        if (A.dsum) {
          float f[VEC];
          load_vec<DT, VEC>(row_of<DT>(A.dsum, row, A.ld_dsum), k, f);
#pragma unroll
          for (int j = 0; j < VEC; ++j) o[j] += f[j];
        }
        store_vec<DT, VEC>(row_of<DT>(A.dx, row, A.ld_dx), k, o);
      }
    }
  }
  float* out = A.partial + (int64_t)blockIdx.x * A.cols;
  if (T > 32) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * T + t < nv)
#pragma unroll
        for (int j = 0; j < VEC; ++j) out[(i * T + t) * VEC + j] = acc[i][j];
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i * T + t < nv)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s_gain[threadIdx.y * A.cols + (i * T + t) * VEC + j] = acc[i][j];
  __syncthreads();
  for (int c = threadIdx.y * T + t; c < A.cols; c += T * blockDim.y) {
    float v = 0.0f;
    for (int y = 0; y < blockDim.y; ++y) v += s_gain[y * A.cols + c];
    out[c] = v;
  }
}

// Longer rows: each is read twice, and the CTA's row of `partial` holds its sums.
template <int DT, int VEC>
__global__ void __launch_bounds__(kMaxT) rmsnorm_bwd_long_kernel(const __grid_constant__ BwdArgs A) {
  __shared__ float2 part[2][32];
  const int T = blockDim.x, t = threadIdx.x;
  const int nv = A.cols / VEC;
  float* out = A.partial + (int64_t)blockIdx.x * A.cols;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x, flip ^= 1) {
    const void* hp = row_of<DT>(A.h, row, A.ld_h);
    const void* dp = row_of<DT>(A.dy, row, A.ld_dy);
    float2 s = make_float2(0.0f, 0.0f);
    for (int k = t; k < nv; k += T) {
      float h[VEC], d[VEC], g[VEC];
      load_vec<DT, VEC>(hp, k, h);
      load_vec<DT, VEC>(dp, k, d);
      load_gain<VEC>(A.gain, k, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        s.x = fmaf(h[j], h[j], s.x);
        s.y = fmaf(d[j] * g[j], h[j], s.y);
      }
    }
    s = row_sum2(s, T, part[flip]);
    const float inv = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(s.x, A.inv_cols, A.eps)));
    const float c = s.y * A.inv_cols * inv * inv;
    const bool first = row == blockIdx.x;
    for (int k = t; k < nv; k += T) {
      float h[VEC], d[VEC], g[VEC], o[VEC];
      load_vec<DT, VEC>(hp, k, h);
      load_vec<DT, VEC>(dp, k, d);
      load_gain<VEC>(A.gain, k, g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        o[j] = inv * (d[j] * g[j] - h[j] * c);
        const float v = d[j] * (h[j] * inv);
        float* a = out + (int64_t)k * VEC + j;
        *a = first ? v : *a + v;   // this thread's column in every row
      }
      if (A.dsum) {
        float f[VEC];
        load_vec<DT, VEC>(row_of<DT>(A.dsum, row, A.ld_dsum), k, f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] += f[j];
      }
      store_vec<DT, VEC>(row_of<DT>(A.dx, row, A.ld_dx), k, o);
    }
  }
}

// dgain[c] = sum of n rows of partial, in an order that n alone fixes.
__global__ void __launch_bounds__(1024) dgain_kernel(const float* partial, int32_t n, int32_t cols, float* dgain) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.0f;
  if (c < cols)
    for (int r = threadIdx.y; r < n; r += 32) v += partial[(int64_t)r * cols + c];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = s[threadIdx.x][threadIdx.y];   // a warp per column
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int cc = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && cc < cols) dgain[cc] = v;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool is_dtype(int v) { return v == QMUON_BF16 || v == QMUON_FP16 || v == QMUON_FP32; }

// Threads of a row and vectors per thread for nv vectors; V == 0: a long row.
struct Shape {
  int T, V;
  int rows_per_cta() const { return T >= 256 || T > 32 ? 1 : 256 / T; }
};

Shape pick_shape(int nv, const int* vs, int n_vs, int min_t, int want_v) {
  for (int i = 0; i < n_vs; ++i) {
    const int V = vs[i];
    if (V < want_v && i + 1 < n_vs) continue;
    int T = (nv + V - 1) / V;
    if (T <= 32) {
      int p = min_t;
      while (p < T) p *= 2;
      T = p;
    } else {
      T = (T + 31) / 32 * 32;
    }
    if (T <= kMaxT) return {T, V};
  }
  return {kMaxT, 0};
}

int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms;
}

template <int DT, int VEC, bool MX>
void launch_fwd(const FwdArgs& A, cudaStream_t s) {
  const int nv = A.cols / VEC;
  static const int vs16[] = {1, 2, 4}, vs1[] = {1, 4, 8};
  const int min_t = !MX ? 1 : VEC == 1 ? 32 : 32 / VEC;
  const Shape S = VEC == 1 ? pick_shape(nv, vs1, 3, min_t, 8) : pick_shape(nv, vs16, 3, min_t, 4);
  const dim3 block(S.T, S.rows_per_cta());
  const int64_t groups = (A.rows + block.y - 1) / block.y;
  const unsigned grid = (unsigned)std::min<int64_t>(groups, ((int64_t)1 << 31) - 1);
  if (S.V == 0) rmsnorm_fwd_long_kernel<DT, VEC, MX><<<grid, block, 0, s>>>(A);
  else if (S.V == 1) rmsnorm_fwd_kernel<DT, VEC, 1, MX><<<grid, block, 0, s>>>(A);
  else if constexpr (VEC == 1) {
    if (S.V == 4) rmsnorm_fwd_kernel<DT, VEC, 4, MX><<<grid, block, 0, s>>>(A);
    else rmsnorm_fwd_kernel<DT, VEC, 8, MX><<<grid, block, 0, s>>>(A);
  } else {
    if (S.V == 2) rmsnorm_fwd_kernel<DT, VEC, 2, MX><<<grid, block, 0, s>>>(A);
    else rmsnorm_fwd_kernel<DT, VEC, 4, MX><<<grid, block, 0, s>>>(A);
  }
}

template <int DT>
void launch_fwd_dt(const FwdArgs& A, bool vec, cudaStream_t s) {
  constexpr int K = Vec16<DT>::kElems;
  if (A.payload) {
    if (vec) launch_fwd<DT, K, true>(A, s);
    else launch_fwd<DT, 1, true>(A, s);
  } else {
    if (vec) launch_fwd<DT, K, false>(A, s);
    else launch_fwd<DT, 1, false>(A, s);
  }
}

// CTAs of the backward pass: one row of `partial` each.
constexpr int kBwdPerSm = 4;
int bwd_grid(int64_t rows, int sms) { return (int)std::min<int64_t>(std::max<int64_t>(rows, 1), (int64_t)sms * kBwdPerSm); }

template <int DT, int VEC>
int launch_bwd(const BwdArgs& A, int sms, cudaStream_t s) {
  const int nv = A.cols / VEC;
  static const int vs16[] = {1, 2, 4}, vs1[] = {1, 4, 8};
  const Shape S = VEC == 1 ? pick_shape(nv, vs1, 3, 1, 4) : pick_shape(nv, vs16, 3, 1, 2);
  const bool too_wide = S.V * VEC >= 16 && S.T > 512;
  const dim3 block(S.T, S.rows_per_cta());
  const int64_t groups = (A.rows + block.y - 1) / block.y;
  const int grid = bwd_grid(groups, sms);
  const size_t smem = S.T > 32 ? 0 : (size_t)block.y * A.cols * 4;
  if (S.V == 0 || too_wide) rmsnorm_bwd_long_kernel<DT, VEC><<<bwd_grid(A.rows, sms), kMaxT, 0, s>>>(A);
  else if (S.V == 1) rmsnorm_bwd_kernel<DT, VEC, 1><<<grid, block, smem, s>>>(A);
  else if constexpr (VEC == 1) {
    if (S.V == 4) rmsnorm_bwd_kernel<DT, VEC, 4><<<grid, block, smem, s>>>(A);
    else rmsnorm_bwd_kernel<DT, VEC, 8><<<grid, block, smem, s>>>(A);
  } else {
    if (S.V == 2) rmsnorm_bwd_kernel<DT, VEC, 2><<<grid, block, smem, s>>>(A);
    else rmsnorm_bwd_kernel<DT, VEC, 4><<<grid, block, smem, s>>>(A);
  }
  return (S.V == 0 || too_wide) ? bwd_grid(A.rows, sms) : grid;
}

// A matrix argument: non-null, aligned to its elements, rows at least cols
// apart; `vec` stays true if every row starts on a 16-byte boundary.
bool check_matrix(const void* p, int64_t ld, int64_t cols, int dt, bool* vec) {
  const size_t es = elem_size(dt);
  if (!p || ld < cols || !is_aligned(p, es)) return false;
  if (!is_aligned(p, 16) || (ld * (int64_t)es) % 16) *vec = false;
  return true;
}

bool check_sizes(int64_t rows, int64_t cols, int dt, float eps) {
  return rows >= 0 && cols >= 1 && cols <= ((int64_t)1 << 30) && rows <= ((int64_t)1 << 40) / cols && is_dtype(dt) &&
         std::isfinite(eps) && eps >= 0.0f;
}

}  // namespace
}  // namespace qm

using namespace qm;

extern "C" qmuon_status qmuon_rmsnorm_forward(const qmuon_rmsnorm* n, void* stream) {
  NvtxRange nvtx_range("qmuon_rmsnorm_forward");
  if (!n || !check_sizes(n->rows, n->cols, n->dtype, n->eps)) return QMUON_ERR_INVALID_ARGUMENT;
  if ((!n->y && !n->payload) || (n->payload == nullptr) != (n->scale_inv == nullptr)) return QMUON_ERR_INVALID_ARGUMENT;
  if (n->payload && n->cols % QMUON_SCALE_BLOCK) return QMUON_ERR_UNSUPPORTED;
  bool vec = n->cols % (16 / elem_size(n->dtype)) == 0 && is_aligned(n->gain, 16) && is_aligned(n->payload, 8);
  if (!n->gain || !is_aligned(n->gain, 4) || !check_matrix(n->x, n->ld_x, n->cols, n->dtype, &vec))
    return QMUON_ERR_INVALID_ARGUMENT;
  if (n->residual && !check_matrix(n->residual, n->ld_residual, n->cols, n->dtype, &vec)) return QMUON_ERR_INVALID_ARGUMENT;
  if (n->sum && !check_matrix(n->sum, n->ld_sum, n->cols, n->dtype, &vec)) return QMUON_ERR_INVALID_ARGUMENT;
  if (n->y && !check_matrix(n->y, n->ld_y, n->cols, n->dtype, &vec)) return QMUON_ERR_INVALID_ARGUMENT;
  if (n->rows == 0) return QMUON_OK;
  FwdArgs A{n->x,    n->residual,    n->gain,   n->sum,  n->y,    n->payload, n->scale_inv, n->rows,
            n->ld_x, n->ld_residual, n->ld_sum, n->ld_y, (int32_t)n->cols, n->eps,    1.0f / (float)n->cols};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n->dtype == QMUON_BF16) launch_fwd_dt<QMUON_BF16>(A, vec, s);
  else if (n->dtype == QMUON_FP16) launch_fwd_dt<QMUON_FP16>(A, vec, s);
  else launch_fwd_dt<QMUON_FP32>(A, vec, s);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? QMUON_OK : set_error("qmuon_rmsnorm_forward (launch)", e);
}

extern "C" size_t qmuon_rmsnorm_workspace_size(int64_t rows, int64_t cols) {
  if (!check_sizes(rows, cols, QMUON_FP32, 0.0f)) return 0;
  const int sms = device_sms();
  return ((size_t)bwd_grid(rows, sms > 0 ? sms : 1) * (size_t)cols * 4 + 255) / 256 * 256;
}

extern "C" qmuon_status qmuon_rmsnorm_backward(const qmuon_rmsnorm_grad* n, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("qmuon_rmsnorm_backward");
  if (!n || !check_sizes(n->rows, n->cols, n->dtype, n->eps)) return QMUON_ERR_INVALID_ARGUMENT;
  bool vec = n->cols % (16 / elem_size(n->dtype)) == 0 && is_aligned(n->gain, 16);
  if (!n->gain || !is_aligned(n->gain, 4) || !n->dgain || !is_aligned(n->dgain, 4) || !ws || !is_aligned(ws, 256))
    return QMUON_ERR_INVALID_ARGUMENT;
  if (!check_matrix(n->dy, n->ld_dy, n->cols, n->dtype, &vec) || !check_matrix(n->h, n->ld_h, n->cols, n->dtype, &vec) ||
      !check_matrix(n->dx, n->ld_dx, n->cols, n->dtype, &vec))
    return QMUON_ERR_INVALID_ARGUMENT;
  if (n->dsum && !check_matrix(n->dsum, n->ld_dsum, n->cols, n->dtype, &vec)) return QMUON_ERR_INVALID_ARGUMENT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n->rows == 0) {
    const cudaError_t e = cudaMemsetAsync(n->dgain, 0, (size_t)n->cols * 4, s);
    return e == cudaSuccess ? QMUON_OK : set_error("qmuon_rmsnorm_backward (memset)", e);
  }
  const int sms = device_sms();
  if (sms <= 0) return set_error_msg("qmuon_rmsnorm_backward: SM count query failed", QMUON_ERR_CUDA);
  if (ws_bytes < qmuon_rmsnorm_workspace_size(n->rows, n->cols)) return QMUON_ERR_WORKSPACE_TOO_SMALL;
  BwdArgs A{n->dy,   n->h,    n->dsum,    n->gain,  n->dx,            static_cast<float*>(ws), n->rows,
            n->ld_dy, n->ld_h, n->ld_dsum, n->ld_dx, (int32_t)n->cols, n->eps,                  1.0f / (float)n->cols};
  constexpr int kHalf = 8, kFull = 4;   // elements of a 16-byte vector
  int grid = 0;
  if (n->dtype == QMUON_BF16) grid = vec ? launch_bwd<QMUON_BF16, kHalf>(A, sms, s) : launch_bwd<QMUON_BF16, 1>(A, sms, s);
  else if (n->dtype == QMUON_FP16) grid = vec ? launch_bwd<QMUON_FP16, kHalf>(A, sms, s) : launch_bwd<QMUON_FP16, 1>(A, sms, s);
  else grid = vec ? launch_bwd<QMUON_FP32, kFull>(A, sms, s) : launch_bwd<QMUON_FP32, 1>(A, sms, s);
  dgain_kernel<<<(unsigned)((n->cols + 31) / 32), dim3(32, 32), 0, s>>>(A.partial, grid, A.cols, n->dgain);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? QMUON_OK : set_error("qmuon_rmsnorm_backward (launch)", e);
}
