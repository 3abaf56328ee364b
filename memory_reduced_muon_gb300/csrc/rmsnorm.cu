// RMS norm with the residual's addition, forward (same-type or MXFP8 output)
// and backward.
//
//   h = x + residual          y = h / sqrt(mean(h^2) + eps) * gain
//   a = dy * gain, n = h inv: dx = inv (a - n mean(a n)) + dsum
//                             dgain = sum over rows of dy n
//
// A row belongs to T threads: a power of two up to a warp (and a CTA then takes
// several rows), or whole warps.  Rows that fit their threads' registers cross
// HBM once: in 16-byte vectors where all arrays' rows start on 16 bytes ("rows"
// kernels), else in pairs of 16-bit elements or single elements ("pieces") or
// by way of shared memory ("staged").  Longer ones are walked twice, the second
// time out of the caches ("walk").
#include <algorithm>
#include <atomic>
#include <cmath>
#include <initializer_list>
#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>
#include <utility>

#include "qm_elem.h"

namespace qm {
namespace {

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
  int32_t align;          // bytes on which all rows start, and which divide a row: 2 (4 for fp32), 4, 8 or 16
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
  int32_t align;          // bytes on which all rows start, and which divide a row: 2 (4 for fp32), 4, 8 or 16
  float eps, inv_cols;
};

template <int DT, class P>
__device__ __forceinline__ auto row_of(P* base, int64_t row, int64_t ld) {
  using B = std::conditional_t<std::is_const_v<P>, const unsigned char, unsigned char>;
  return static_cast<B*>(base) + row * ld * elem_size(DT);
}

// Sum of v over the T threads of a row, the same bits in all of them.  T > 32:
// `part` is one value per warp of the CTA; callers alternate two of them, so
// that one barrier per sum is enough.  MANY: the CTA may have several rows of
// more than a warp, each with a barrier of its own (a kernel that names its
// barriers at run time reserves all sixteen, which leaves an SM few CTAs).
__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ float2 plus(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float lane_xor(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
__device__ __forceinline__ float2 lane_xor(float2 v, int o) { return make_float2(lane_xor(v.x, o), lane_xor(v.y, o)); }

template <bool MANY, class S>
__device__ __forceinline__ S row_sum(S v, int T, S* part) {
  if (T >= 32) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = plus(v, lane_xor(v, o));
  } else {
    for (int o = T >> 1; o > 0; o >>= 1) v = plus(v, lane_xor(v, o));
  }
  if (T <= 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = T >> 5;
  if constexpr (MANY) part += threadIdx.y * nw;
  if (lane == 0) part[warp] = v;
  if constexpr (MANY) asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(T) : "memory");
  else __syncthreads();
  v = lane < nw ? part[lane] : S{};
  for (int o = 16; o > 0; o >>= 1) v = plus(v, lane_xor(v, o));
  return v;
}

__device__ __forceinline__ float inverse_norm(float sumsq, float inv_cols, float eps) {
  return rsqrtf(fmaf(sumsq, inv_cols, eps));   // 2 ulp
}

// The MXFP8 codes of N values held by a thread whose neighbours hold the rest
// of the 32-element block; every thread of the warp calls it.
template <int N>
__device__ __forceinline__ void store_mxfp8(const float* y, bool valid, int64_t e, uint8_t* payload, uint8_t* scale) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) amax = fmaxf(amax, fabsf(y[j]));
  if (!valid) amax = 0.0f;
  if constexpr (N == 1) {
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));   // not negative: ordered as integers
  } else {
#pragma unroll
    for (int o = 16 / N; o > 0; o >>= 1) amax = fmaxf(amax, lane_xor(amax, o));
  }
  const int byte = e8m0_of_amax(amax);
  const float mult = pow2_from_e8m0(byte);
  if (!valid) return;
  if constexpr (N == 1) {
    payload[e] = (uint8_t)cvt_e4m3x2(__fmul_rn(y[0], mult), 0.0f);
  } else if constexpr (N == 2) {
    const uint32_t w = cvt_e4m3x2(__fmul_rn(y[0], mult), __fmul_rn(y[1], mult));
    if ((reinterpret_cast<uintptr_t>(payload) & 1) == 0) *reinterpret_cast<uint16_t*>(payload + e) = (uint16_t)w;
    else payload[e] = (uint8_t)w, payload[e + 1] = (uint8_t)(w >> 8);
  } else {
    uint32_t w[N / 4];
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      const float2 a = mul2_rn(make_float2(y[4 * j], y[4 * j + 1]), mult), b = mul2_rn(make_float2(y[4 * j + 2], y[4 * j + 3]), mult);
      w[j] = cvt_e4m3x2(a.x, a.y) | (cvt_e4m3x2(b.x, b.y) << 16);
    }
    if constexpr (N == 8) *reinterpret_cast<uint2*>(payload + e) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(payload + e) = w[0];
  }
  if ((e & 31) == 0) scale[e >> 5] = (uint8_t)byte;
}

// ---------------------------------------------------------------------------
// rows that start anywhere, in shared memory
// ---------------------------------------------------------------------------
// The 16-byte words of memory that hold a row are copied to a slot as they lie
// there, so that the row starts in its slot where it starts in its word; the
// words at an array's two ends, of which a part is not the array's, come by
// elements.  Threads then read pairs of columns, the same ones in every row
// whatever its start.
template <bool MANY>   // see row_sum
__device__ __forceinline__ void row_sync(int T) {
  if (T <= 32) __syncwarp();
  else if constexpr (MANY) asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(T) : "memory");
  else __syncthreads();
}

__host__ __device__ constexpr int slot_bytes(int cols, int es) { return (cols * es + 15) / 16 * 16 + 16; }

// An array's first byte and the one after its last, between which words are read whole.
struct Extent {
  const unsigned char *begin, *end;
};
template <int DT>
__device__ __forceinline__ Extent extent_of(const void* p, int64_t rows, int64_t ld, int cols) {
  const unsigned char* b = static_cast<const unsigned char*>(p);
  return {b, b + ((rows - 1) * ld + cols) * elem_size(DT)};
}

template <int DT>
__device__ __forceinline__ void stage_row(unsigned char* slot, const Extent& E, const unsigned char* row, int cols, int t, int T) {
  constexpr int es = elem_size(DT);
  const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15), end = off + cols * es, last = (end - 1) >> 4;
  const unsigned char* words = row - off;
  const int from = words < E.begin, to = last - (words + 16 * last + 16 > E.end);
  const unsigned char* w = words + 16 * t;
  unsigned char* d = slot + 16 * t;
  for (int j = t; j <= to; j += T, w += 16 * T, d += 16 * T)
    if (j >= from) async16(d, w);
  if (from + last > to) {   // a word at the array's start or end
    for (int b = t * es; b < end; b += T * es)
      if (b >= off && (b < 16 * from || b >= 16 * to + 16)) {
        if constexpr (es == 2) *reinterpret_cast<uint16_t*>(slot + b) = *reinterpret_cast<const uint16_t*>(words + b);
        else *reinterpret_cast<uint32_t*>(slot + b) = *reinterpret_cast<const uint32_t*>(words + b);
      }
  }
}

// V pairs of columns of a staged row: 16-bit ones side by side, T pairs apart;
// fp32 ones T columns apart.
template <int DT, int V>
struct Pairs {
  using Raw = std::conditional_t<DT == QMUON_FP32, float2, uint32_t>;
  __device__ __forceinline__ static int col(int i, int half, int t, int T) {
    return DT == QMUON_FP32 ? t + (2 * i + half) * T : 2 * (t + i * T) + half;
  }
  // `row`: the low bits of where the row starts in memory
  __device__ __forceinline__ static void load(const unsigned char* slot, uint32_t row, int cols, int t, int T, Raw* r) {
    const int off = (int)(row & 15);
    if constexpr (DT == QMUON_FP32) {
      const float* p = reinterpret_cast<const float*>(slot + off);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int a = col(i, 0, t, T), b = col(i, 1, t, T);
        r[i] = make_float2(a < cols ? p[a] : 0.0f, b < cols ? p[b] : 0.0f);
      }
    } else {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(slot + (off & ~3)) + t;
      const int n = (cols + 1) >> 1;
      if (off & 2) {
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] = t + i * T < n ? __byte_perm(p[i * T], p[i * T + 1], 0x5432u) : 0u;
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] = t + i * T < n ? p[i * T] : 0u;
      }
      if (cols & 1) {   // an odd row's last
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (t + i * T == cols >> 1) r[i] &= 0xFFFFu;
      }
    }
  }
  __device__ __forceinline__ static float2 unpack(Raw r) {
    if constexpr (DT == QMUON_FP32) return r;
    else return unpack2<DT>(r);
  }
  __device__ __forceinline__ static void store(unsigned char* row, int cols, int t, int T, const float2* f) {
    if constexpr (DT == QMUON_FP32) {
      float* p = reinterpret_cast<float*>(row);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int a = col(i, 0, t, T), b = col(i, 1, t, T);
        if (a < cols) p[a] = f[i].x;
        if (b < cols) p[b] = f[i].y;
      }
    } else {
      const int n = cols >> 1;
      uint16_t* p = reinterpret_cast<uint16_t*>(row) + 2 * t;
      uint32_t w[V];
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = pack2<DT>(f[i].x, f[i].y);
      if ((reinterpret_cast<uintptr_t>(row) & 2) == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (t + i * T < n) *reinterpret_cast<uint32_t*>(p + 2 * i * T) = w[i];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (t + i * T < n) p[2 * i * T] = (uint16_t)w[i], p[2 * i * T + 1] = (uint16_t)(w[i] >> 16);
      }
      if (cols & 1) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (t + i * T == n) p[2 * i * T] = (uint16_t)w[i];
      }
    }
  }
};

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// blockDim = (T, rows per CTA); V 16-byte vectors per thread, those of x and of
// the residual all in flight before the first is unpacked (unpacking x first, with
// unpaired arithmetic, took 98 us for the second figure).  One CTA per row, or per
// 256 threads of short rows: bound by DRAM, 16384 x 4096 bf16 with the residual
// to bf16 80 us (6.7 TB/s), to MXFP8 70 us (6.8 TB/s); 131072 x 128 bf16 14 us.
constexpr int fwd_max_threads(int V) { return V == 4 ? 512 : 1024; }

template <int DT, int V, bool RES, bool MX>
__global__ void __launch_bounds__(fwd_max_threads(V)) rmsnorm_fwd_rows_kernel(const __grid_constant__ FwdArgs A) {
  using X = Vec16<DT>;
  constexpr int P = X::kPairs;
  __shared__ float part[2][32];
  const int T = blockDim.x, t = threadIdx.x;
  const int nv = A.cols / X::kElems;
  depends_wait();
  int flip = 0;
  // every thread of a warp leaves the loop together: the CTA's rows of one pass are one step of it
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < A.rows; r0 += (int64_t)gridDim.x * blockDim.y, flip ^= 1) {
    const int64_t row = r0 + threadIdx.y;
    const int n = row < A.rows ? nv : 0;
    const uint4* x = reinterpret_cast<const uint4*>(row_of<DT>(A.x, row, A.ld_x)) + t;
    const uint4* res = reinterpret_cast<const uint4*>(row_of<DT>(A.residual, row, A.ld_residual)) + t;
    uint4 rx[V], rr[RES ? V : 1];
#pragma unroll
    for (int i = 0; i < V; ++i) rx[i] = i * T + t < n ? x[i * T] : make_uint4(0, 0, 0, 0);
    if constexpr (RES)
#pragma unroll
      for (int i = 0; i < V; ++i) rr[i] = i * T + t < n ? res[i * T] : make_uint4(0, 0, 0, 0);
    float2 h[V][P], ss = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      X::unpack(rx[i], h[i]);
      if constexpr (RES) {
        float2 f[P];
        X::unpack(rr[i], f);
#pragma unroll
        for (int j = 0; j < P; ++j) h[i][j] = add2(h[i][j], f[j]);
      }
#pragma unroll
      for (int j = 0; j < P; ++j) ss = fma2(h[i][j], h[i][j], ss);
    }
    // The gain of each vector comes before the output of the one before it is stored, and the first one's before the
    // sum: its way from memory may be as long as the row's.
    const float4* gain = reinterpret_cast<const float4*>(A.gain) + t * (P / 2);
    float4 g[P / 2];
    auto load_gain = [&](int i) {
#pragma unroll
      for (int j = 0; j < P / 2; ++j) g[j] = i * T + t < n ? gain[i * T * (P / 2) + j] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };
    load_gain(0);
    if (A.sum) {
      uint4* sum = reinterpret_cast<uint4*>(row_of<DT>(A.sum, row, A.ld_sum)) + t;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i * T + t < n) sum[i * T] = X::pack(h[i]);
    }
    const float inv = inverse_norm(row_sum<false>(ss.x + ss.y, T, part[flip]), A.inv_cols, A.eps);
    uint4* y = reinterpret_cast<uint4*>(row_of<DT>(A.y, row, A.ld_y)) + t;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool in = i * T + t < n;
      if (in) {
#pragma unroll
        for (int j = 0; j < P / 2; ++j) {
          h[i][2 * j] = mul2_rn(mul2_rn(h[i][2 * j], inv), make_float2(g[j].x, g[j].y));
          h[i][2 * j + 1] = mul2_rn(mul2_rn(h[i][2 * j + 1], inv), make_float2(g[j].z, g[j].w));
        }
      }
      if (i + 1 < V) load_gain(i + 1);
      if (in && (!MX || A.y)) y[i * T] = X::pack(h[i]);
      if constexpr (MX)
        store_mxfp8<2 * P>(reinterpret_cast<const float*>(h[i]), in, row * A.cols + (int64_t)(i * T + t) * X::kElems, A.payload,
                           A.scale);
    }
  }
}

// A row whose arrays are not aligned, in pieces of one element or, where all
// arrays' rows start alike within 4 bytes, of a pair of 16-bit elements; these
// start at column `head` (0 or 1) and leave one element at either end, which
// the first and the last thread hold besides, loaded with the others (loaded
// after them they cost another trip to memory).  Bound by its instructions, 37
// per element, three quarters of what the schedulers can issue: 6001 x 2049 fp16
// with an odd stride 20.8 us, 0.70 of the copy rate (41.7 us by single elements
// that were read twice).
template <int DT, int N>
struct Piece {
  using Raw = std::conditional_t<N == 2 || DT == QMUON_FP32, uint32_t, uint16_t>;
  [[maybe_unused]] static constexpr int kStep = 32 * N;   // columns between a thread's pieces: a warp's lie side by side
  __device__ __forceinline__ static Raw load(const unsigned char* row, int c) {
    return *reinterpret_cast<const Raw*>(row + c * elem_size(DT));
  }
  __device__ __forceinline__ static float2 unpack(Raw w) {
    if constexpr (N == 2) return unpack2<DT>(w);
    else if constexpr (DT == QMUON_FP32) return make_float2(__uint_as_float(w), 0.0f);
    else return make_float2(unpack2<DT>(w).x, 0.0f);
  }
  __device__ __forceinline__ static void store(unsigned char* row, int c, float2 f) {
    if constexpr (N == 2) *reinterpret_cast<uint32_t*>(row + c * 2) = pack2<DT>(f.x, f.y);
    else store_elem<DT>(row, c, f.x);
  }
};

// A thread has P pieces: piece i is 32 i on from its first one, so that a warp's
// lie side by side.
template <int P>
__device__ __forceinline__ int first_piece(int t) {
  return (t >> 5) * (32 * P) + (t & 31);
}

template <int DT, int N, int P, bool RES>
__global__ void __launch_bounds__(1024) rmsnorm_fwd_pieces_kernel(const __grid_constant__ FwdArgs A) {
  using One = Piece<DT, 1>;
  using Some = Piece<DT, N>;
  __shared__ float part[2][32];
  const int T = blockDim.x, t = threadIdx.x;
  depends_wait();
  int flip = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < A.rows; r0 += (int64_t)gridDim.x * blockDim.y, flip ^= 1) {
    const int64_t row = r0 + threadIdx.y;
    const bool live = row < A.rows;
    const unsigned char* x = row_of<DT>(A.x, row, A.ld_x);
    const unsigned char* res = row_of<DT>(A.residual, row, A.ld_residual);
    const int head = N == 2 ? (int)(reinterpret_cast<uintptr_t>(x) >> 1) & 1 : 0;
    const int n = live ? (A.cols - head) / N : 0;   // whole pieces, from column head on
    // the single elements of the first and the last thread (one thread's, where T is 1: never, T is 32 or more)
    const int edge = N == 1 || !live         ? -1
                     : t == 0 && head        ? 0
                     : t == T - 1 && ((A.cols - head) & 1) ? A.cols - 1
                                             : -1;
    typename Some::Raw rx[P], rr[RES ? P : 1];
    typename One::Raw ex = 0, er = 0;
    if (edge >= 0) {
      ex = One::load(x, edge);
      if constexpr (RES) er = One::load(res, edge);
    }
    const int k0 = first_piece<P>(t), c0 = head + N * k0;
    x += c0 * elem_size(DT);
    res += c0 * elem_size(DT);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      rx[i] = k0 + 32 * i < n ? Some::load(x, i * Some::kStep) : 0;
      if constexpr (RES) rr[i] = k0 + 32 * i < n ? Some::load(res, i * Some::kStep) : 0;
    }
    float2 h[P], ss = make_float2(0.0f, 0.0f);
    float he = One::unpack(ex).x;
    if constexpr (RES) he += One::unpack(er).x;
    ss.x = he * he;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      h[i] = Some::unpack(rx[i]);
      if constexpr (RES) h[i] = add2(h[i], Some::unpack(rr[i]));
      ss = fma2(h[i], h[i], ss);
    }
    const float* gain = A.gain + c0;
    auto gain_of = [&](int i) {
      const int d = i * Some::kStep;
      return make_float2(gain[d], N == 2 ? gain[d + N - 1] : 0.0f);
    };
    const float ge = edge >= 0 ? A.gain[edge] : 0.0f;
    const float inv = inverse_norm(row_sum<false>(ss.x + ss.y, T, part[flip]), A.inv_cols, A.eps);
    unsigned char* sum = row_of<DT>(A.sum, row, A.ld_sum);
    unsigned char* y = row_of<DT>(A.y, row, A.ld_y);
    if (edge >= 0) {
      if (A.sum) One::store(sum, edge, make_float2(he, 0.0f));
      One::store(y, edge, make_float2(he * inv * ge, 0.0f));
    }
    sum += c0 * elem_size(DT);
    y += c0 * elem_size(DT);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const bool in = k0 + 32 * i < n;
      const int d = i * Some::kStep;
      if (in) {
        const float2 g = gain_of(i);
        if (A.sum) Some::store(sum, d, h[i]);
        h[i] = mul2_rn(mul2_rn(h[i], inv), g);
        Some::store(y, d, h[i]);
      }
    }
  }
}

// Rows in a slot each (see above): where 16-bit arrays start unlike each other,
// and to MXFP8, whose blocks of 32 start where pairs of a row with a head do not.
// Bound by its instructions (64 per element, 0.78 issued per cycle and
// scheduler): 8000 x 4096 bf16 with a residual and odd strides to MXFP8 72 us,
// 97 by single elements in registers and 94 with four pairs per thread;
// 9000 x 7001 bf16 with arrays that start unlike each other 145 us, 207.
template <int DT, int V, bool RES, bool MX>
__global__ void __launch_bounds__(1024) rmsnorm_fwd_staged_kernel(const __grid_constant__ FwdArgs A) {
  using X = Pairs<DT, V>;
  __shared__ float part[2][32];
  extern __shared__ __align__(16) unsigned char smem[];
  const int T = blockDim.x, t = threadIdx.x, bytes = slot_bytes(A.cols, elem_size(DT));
  unsigned char* slot = smem + threadIdx.y * (RES ? 2 : 1) * bytes;
  depends_wait();
  const Extent ex = extent_of<DT>(A.x, A.rows, A.ld_x, A.cols), er = extent_of<DT>(A.residual, A.rows, A.ld_residual, A.cols);
  int flip = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < A.rows; r0 += (int64_t)gridDim.x * blockDim.y, flip ^= 1) {
    const int64_t row = r0 + threadIdx.y;
    const int cols = row < A.rows ? A.cols : 0;
    const unsigned char *x = row_of<DT>(A.x, row, A.ld_x), *res = row_of<DT>(A.residual, row, A.ld_residual);
    if (cols) {
      stage_row<DT>(slot, ex, x, cols, t, T);
      if constexpr (RES) stage_row<DT>(slot + bytes, er, res, cols, t, T);
    }
    async_commit();
    float2 gain[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int a = X::col(i, 0, t, T), b = X::col(i, 1, t, T);
      gain[i] = make_float2(a < cols ? A.gain[a] : 0.0f, b < cols ? A.gain[b] : 0.0f);
    }
    async_wait<0>();
    row_sync<false>(T);
    typename X::Raw rx[V], rr[RES ? V : 1];
    X::load(slot, (uint32_t)(uintptr_t)x, cols, t, T, rx);
    if constexpr (RES) X::load(slot + bytes, (uint32_t)(uintptr_t)res, cols, t, T, rr);
    float2 h[V], ss = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      h[i] = X::unpack(rx[i]);
      if constexpr (RES) h[i] = add2(h[i], X::unpack(rr[i]));
      ss = fma2(h[i], h[i], ss);
    }
    const float inv = inverse_norm(row_sum<false>(ss.x + ss.y, T, part[flip]), A.inv_cols, A.eps);
    if (T <= 32) __syncwarp();   // else row_sum's barrier: all threads of the row have read the slots
    if (A.sum) X::store(row_of<DT>(A.sum, row, A.ld_sum), cols, t, T, h);
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = mul2_rn(mul2_rn(h[i], inv), gain[i]);
    if (!MX || A.y) X::store(row_of<DT>(A.y, row, A.ld_y), cols, t, T, h);
    if constexpr (MX) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int a = X::col(i, 0, t, T), b = X::col(i, 1, t, T);
        const int64_t e = row * A.cols;
        if constexpr (DT == QMUON_FP32) {
          store_mxfp8<1>(&h[i].x, a < cols, e + a, A.payload, A.scale);
          store_mxfp8<1>(&h[i].y, b < cols, e + b, A.payload, A.scale);
        } else {
          store_mxfp8<2>(&h[i].x, a < cols, e + a, A.payload, A.scale);
        }
      }
    }
  }
}

// N consecutive elements of a row at column c, moved at once: one, or 4, 8 or
// 16 bytes of them.
template <int DT, int N>
__device__ __forceinline__ void load_n(const void* row, int c, float* f) {
  constexpr int kBytes = N * elem_size(DT);
  const void* p = static_cast<const unsigned char*>(row) + (int64_t)c * elem_size(DT);
  if constexpr (N == 1) {
    f[0] = load_elem<DT>(p, 0);
  } else {
    uint32_t w[kBytes / 4];
    if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(w) = *static_cast<const uint4*>(p);
    else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(w) = *static_cast<const uint2*>(p);
    else w[0] = *static_cast<const uint32_t*>(p);
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i) {
      if constexpr (DT == QMUON_FP32) f[i] = __uint_as_float(w[i]);
      else reinterpret_cast<float2*>(f)[i] = unpack2<DT>(w[i]);
    }
  }
}
template <int DT, int N>
__device__ __forceinline__ void store_n(void* row, int c, const float* f) {
  constexpr int kBytes = N * elem_size(DT);
  void* p = static_cast<unsigned char*>(row) + (int64_t)c * elem_size(DT);
  if constexpr (N == 1) {
    store_elem<DT>(p, 0, f[0]);
  } else {
    uint32_t w[kBytes / 4];
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i) {
      if constexpr (DT == QMUON_FP32) w[i] = __float_as_uint(f[i]);
      else w[i] = pack2<DT>(f[2 * i], f[2 * i + 1]);
    }
    if constexpr (kBytes == 16) *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kBytes == 8) *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *static_cast<uint32_t*>(p) = w[0];
  }
}

// N fp32 values side by side, N of the gain or of its gradient.
template <int N>
__device__ __forceinline__ void load_f32(const float* p, float* f) {
  if constexpr (N == 1) f[0] = p[0];
  else if constexpr (N == 2) *reinterpret_cast<float2*>(f) = *reinterpret_cast<const float2*>(p);
  else
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(f + i) = *reinterpret_cast<const float4*>(p + i);
}
template <int N>
__device__ __forceinline__ void store_f32(float* p, const float* f) {
  if constexpr (N == 1) p[0] = f[0];
  else if constexpr (N == 2) *reinterpret_cast<float2*>(p) = *reinterpret_cast<const float2*>(f);
  else
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = *reinterpret_cast<const float4*>(f + i);
}

// Rows longer than a CTA holds: read for the sum, and again, out of the
// caches, for the output.
template <int DT, int N, bool MX>
__global__ void __launch_bounds__(1024) rmsnorm_fwd_walk_kernel(const __grid_constant__ FwdArgs A) {
  __shared__ float part[2][32];
  const int T = blockDim.x, t = threadIdx.x;
  depends_wait();
  int flip = 0;
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x, flip ^= 1) {
    const void* x = row_of<DT>(A.x, row, A.ld_x);
    const void* res = row_of<DT>(A.residual, row, A.ld_residual);
    auto load = [&](int c, float* h) {
      load_n<DT, N>(x, c, h);
      if (A.residual) {
        float f[N];
        load_n<DT, N>(res, c, f);
#pragma unroll
        for (int j = 0; j < N; ++j) h[j] += f[j];
      }
    };
    float ss = 0.0f;
#pragma unroll 4
    for (int c = t * N; c < A.cols; c += T * N) {
      float h[N];
      load(c, h);
#pragma unroll
      for (int j = 0; j < N; ++j) ss = fmaf(h[j], h[j], ss);
    }
    const float inv = inverse_norm(row_sum<false>(ss, T, part[flip]), A.inv_cols, A.eps);
#pragma unroll 2
    for (int c0 = 0; c0 < A.cols; c0 += T * N) {   // the same number of passes in every thread: lanes share scales
      const int c = c0 + t * N;
      float h[N] = {};
      if (c < A.cols) {
        load(c, h);
        if (A.sum) store_n<DT, N>(row_of<DT>(A.sum, row, A.ld_sum), c, h);
        float g[N];
        load_f32<N>(A.gain + c, g);
#pragma unroll
        for (int j = 0; j < N; ++j) h[j] = h[j] * inv * g[j];
        if (A.y) store_n<DT, N>(row_of<DT>(A.y, row, A.ld_y), c, h);
      }
      if constexpr (MX) store_mxfp8<N>(h, c < A.cols, row * A.cols + c, A.payload, A.scale);
    }
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// A CTA walks over rows and keeps the gradient of the gain of its threads'
// columns, which leaves as one row of `partial`; dgain_kernel adds those rows
// in order.  The next rows come through a ring of shared-memory slots, each
// thread's own, `stages` rows ahead.  A CTA has to stay for that sum to stay in
// registers.  16384 x 4096 bf16: 81 us with dgain_kernel (6.6 TB/s), 131072 x 128
// fp32 34 us.  CTAs of 8, 16 or 24 rows, whose partial sums are then many, took
// 96 to 99 us for the first.
constexpr int bwd_max_threads(int V) { return V >= 4 ? 512 : 256; }

__device__ __forceinline__ void wait_rows(int pending) {
  if (pending >= 2) async_wait<2>();
  else if (pending == 1) async_wait<1>();
  else async_wait<0>();
}

template <int DT, int V, bool DSUM>
__global__ void __launch_bounds__(bwd_max_threads(V)) rmsnorm_bwd_rows_kernel(const __grid_constant__ BwdArgs A, int stages) {
  using X = Vec16<DT>;
  constexpr int P = X::kPairs;
  constexpr int kArrays = DSUM ? 3 : 2;
  constexpr bool kKeepGain = V <= 4;   // in registers; else read again for each row
  __shared__ float2 part[2][32];
  extern __shared__ __align__(16) unsigned char smem[];
  const int T = blockDim.x, t = threadIdx.x, threads = T * blockDim.y, me = threadIdx.y * T + t;
  depends_wait();
  uint4* ring = reinterpret_cast<uint4*>(smem) + me;   // [stages][kArrays][V][threads]
  const int nv = A.cols / X::kElems;
  const float4* gain = reinterpret_cast<const float4*>(A.gain) + t * (P / 2);
  auto load_gain = [&](int i, float2* g) {
#pragma unroll
    for (int j = 0; j < P; j += 2) {
      const float4 q = i * T + t < nv ? gain[i * T * (P / 2) + j / 2] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      g[j] = make_float2(q.x, q.y);
      g[j + 1] = make_float2(q.z, q.w);
    }
  };
  float2 acc[V][P], kept[kKeepGain ? V : 1][P];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < P; ++j) acc[i][j] = make_float2(0.0f, 0.0f);
    if constexpr (kKeepGain) load_gain(i, kept[i]);
  }
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  auto issue = [&](int64_t row, uint4* slot) {
    if (row < A.rows) {
      const uint4* src[3] = {reinterpret_cast<const uint4*>(row_of<DT>(A.h, row, A.ld_h)),
                             reinterpret_cast<const uint4*>(row_of<DT>(A.dy, row, A.ld_dy)),
                             DSUM ? reinterpret_cast<const uint4*>(row_of<DT>(A.dsum, row, A.ld_dsum)) : nullptr};
#pragma unroll
      for (int a = 0; a < kArrays; ++a)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i * T + t < nv) async16(slot + (a * V + i) * threads, src[a] + i * T + t);
    }
    async_commit();   // one group per row, empty past the end
  };
  const int64_t r0 = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  for (int s = 0; s < stages; ++s) issue(r0 + s * step, ring + s * kArrays * V * threads);
  int flip = 0, s = 0;
  // the same number of passes in every thread of the CTA
  for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < A.rows; base += step, flip ^= 1) {
    const int64_t row = base + threadIdx.y;
    const int n = row < A.rows ? nv : 0;
    uint4* slot = ring + s * kArrays * V * threads;
    wait_rows(stages - 1);
    float2 sh = make_float2(0.0f, 0.0f), sa = sh;   // sums of h^2 and a h
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * T + t < n) {
        float2 h[P], d[P], g[P];
        X::unpack(slot[i * threads], h);
        X::unpack(slot[(V + i) * threads], d);
        if constexpr (!kKeepGain) load_gain(i, g);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          sh = fma2(h[j], h[j], sh);
          sa = fma2(mul2_rn(d[j], kKeepGain ? kept[i % V][j] : g[j]), h[j], sa);
        }
      }
    const float2 sum = row_sum<true>(make_float2(sh.x + sh.y, sa.x + sa.y), T, part[flip]);
    const float inv = inverse_norm(sum.x, A.inv_cols, A.eps);
    const float c = -(sum.y * A.inv_cols * inv * inv);   // -mean(a h) inv^2
    uint4* dx = reinterpret_cast<uint4*>(row_of<DT>(A.dx, row, A.ld_dx)) + t;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * T + t < n) {
        float2 h[P], d[P], o[P], g[P];
        X::unpack(slot[i * threads], h);
        X::unpack(slot[(V + i) * threads], d);
        if constexpr (DSUM) X::unpack(slot[(2 * V + i) * threads], o);
        if constexpr (!kKeepGain) load_gain(i, g);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const float2 a = mul2_rn(d[j], kKeepGain ? kept[i % V][j] : g[j]);
          const float2 e = fma2(h[j], make_float2(c, c), a);
          if constexpr (DSUM) o[j] = fma2(e, make_float2(inv, inv), o[j]);
          else o[j] = mul2_rn(e, inv);
          acc[i][j] = fma2(d[j], mul2_rn(h[j], inv), acc[i][j]);
        }
        dx[i * T] = X::pack(o);
      }
    issue(row + stages * step, slot);
    s = s + 1 == stages ? 0 : s + 1;
  }
  float* out = A.partial + (int64_t)blockIdx.x * A.cols;
  if (blockDim.y == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * T + t < nv)
#pragma unroll
        for (int j = 0; j < P; j += 2)
          reinterpret_cast<float4*>(out)[(i * T + t) * (P / 2) + j / 2] =
              make_float4(acc[i][j].x, acc[i][j].y, acc[i][j + 1].x, acc[i][j + 1].y);
    return;
  }
  async_wait<0>();
  __syncthreads();   // the ring is free
  float* rows = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i * T + t < nv)
#pragma unroll
      for (int j = 0; j < P; ++j)
        *reinterpret_cast<float2*>(rows + (size_t)threadIdx.y * A.cols + (i * T + t) * X::kElems + 2 * j) = acc[i][j];
  __syncthreads();
  for (int k = me; k < A.cols; k += threads) {
    float v = 0.0f;
    for (int y = 0; y < (int)blockDim.y; ++y) v += rows[(size_t)y * A.cols + k];
    out[k] = v;
  }
}

// Unaligned rows of 16-bit elements that start alike in all arrays, in pairs
// (see the forward pass); the next row's are loaded while one is computed.
// Pairs start at column 0 or 1, by the row, so that a thread's columns differ
// between the two kinds of rows: it sums each kind's apart.
constexpr int bwd_piece_threads = 512;

template <int DT, int P, bool DSUM>
__global__ void __launch_bounds__(bwd_piece_threads) rmsnorm_bwd_pieces_kernel(const __grid_constant__ BwdArgs A) {
  using One = Piece<DT, 1>;
  using Some = Piece<DT, 2>;
  __shared__ float2 part[2][32];
  extern __shared__ __align__(16) float s_acc[];   // [rows of the CTA][cols] of sums, then the gain and zeros for all pieces
  const int T = blockDim.x, t = threadIdx.x, k0 = first_piece<P>(t);
  depends_wait();
  float* s_gain = s_acc + (size_t)blockDim.y * A.cols;
  for (int c = threadIdx.y * T + t; c < T * P * 2 + 2; c += T * blockDim.y) s_gain[c] = c < A.cols ? A.gain[c] : 0.0f;
  struct Raw {
    typename Some::Raw h[P], d[P], s[DSUM ? P : 1];
    typename One::Raw he, de, se;
    int head, n, edge;
  };
  auto load = [&](int64_t row, Raw& r) {
    const bool live = row < A.rows;
    const unsigned char* h = row_of<DT>(A.h, row, A.ld_h);
    const unsigned char* d = row_of<DT>(A.dy, row, A.ld_dy);
    const unsigned char* s = row_of<DT>(A.dsum, row, A.ld_dsum);
    r.head = (int)(reinterpret_cast<uintptr_t>(h) >> 1) & 1;
    r.n = live ? (A.cols - r.head) / 2 : 0;
    r.edge = !live                                  ? -1
             : t == 0 && r.head                     ? 0
             : t == T - 1 && ((A.cols - r.head) & 1) ? A.cols - 1
                                                    : -1;
    r.he = r.de = r.se = 0;
    if (r.edge >= 0) {
      r.he = One::load(h, r.edge);
      r.de = One::load(d, r.edge);
      if constexpr (DSUM) r.se = One::load(s, r.edge);
    }
    const int c0 = (r.head + 2 * k0) * 2;
    h += c0, d += c0, s += c0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const bool in = k0 + 32 * i < r.n;
      r.h[i] = in ? Some::load(h, i * Some::kStep) : 0;
      r.d[i] = in ? Some::load(d, i * Some::kStep) : 0;
      if constexpr (DSUM) r.s[i] = in ? Some::load(s, i * Some::kStep) : 0;
    }
  };
  float2 acc[2][P] = {};   // of pairs from column 0, from column 1
  float acc_edge = 0.0f;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  Raw in;
  load((int64_t)blockIdx.x * blockDim.y + threadIdx.y, in);
  __syncthreads();
  int flip = 0;
  for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < A.rows; base += step, flip ^= 1) {
    const int64_t row = base + threadIdx.y;
    Raw next;
    load(row + step, next);
    const float* g0 = s_gain + in.head + 2 * k0;
    auto gain = [&](int i) {
      return make_float2(g0[i * Some::kStep], g0[i * Some::kStep + 1]);
    };
    const float he = One::unpack(in.he).x, de = One::unpack(in.de).x, ge = in.edge >= 0 ? s_gain[in.edge] : 0.0f;
    float2 sh = make_float2(he * he, 0.0f), sa = make_float2(de * ge * he, 0.0f);   // sums of h^2 and a h
#pragma unroll
    for (int i = 0; i < P; ++i) {   // pieces that are not there hold zeros: no branches
      const float2 h = Some::unpack(in.h[i]);
      sh = fma2(h, h, sh);
      sa = fma2(mul2_rn(Some::unpack(in.d[i]), gain(i)), h, sa);
    }
    const float2 sum = row_sum<true>(make_float2(sh.x + sh.y, sa.x + sa.y), T, part[flip]);
    const float inv = inverse_norm(sum.x, A.inv_cols, A.eps);
    const float c = -(sum.y * A.inv_cols * inv * inv);   // -mean(a h) inv^2
    unsigned char* dx = row_of<DT>(A.dx, row, A.ld_dx);
    if (in.edge >= 0) {
      float o = inv * fmaf(he, c, de * ge);
      if constexpr (DSUM) o += One::unpack(in.se).x;
      One::store(dx, in.edge, make_float2(o, 0.0f));
      acc_edge = fmaf(de, he * inv, acc_edge);
    }
    dx += (in.head + 2 * k0) * 2;
    auto finish = [&](float2* sums) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float2 h = Some::unpack(in.h[i]), d = Some::unpack(in.d[i]);
        const float2 e = fma2(h, make_float2(c, c), mul2_rn(d, gain(i)));
        float2 o;
        if constexpr (DSUM) o = fma2(e, make_float2(inv, inv), Some::unpack(in.s[i]));
        else o = mul2_rn(e, inv);
        if (k0 + 32 * i < in.n) Some::store(dx, i * Some::kStep, o);
        sums[i] = fma2(d, mul2_rn(h, inv), sums[i]);
      }
    };
    if (row < A.rows) {   // past the end inv is infinite where eps is zero
      if (in.head == 0) finish(acc[0]);
      else finish(acc[1]);
    }
    in = next;
  }
  // the columns' sums: those of rows whose pairs start at column 0, then at column 1, then the ends'
  float* mine = s_acc + (size_t)threadIdx.y * A.cols;
  for (int c = t; c < A.cols; c += T) mine[c] = 0.0f;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = kind + 2 * (k0 + 32 * i);
      if (c + 2 <= A.cols) {
        mine[c] += acc[kind][i].x;
        mine[c + 1] += acc[kind][i].y;
      }
    }
  }
  __syncthreads();
  if (t == 0) mine[0] += acc_edge;
  __syncthreads();   // one column: both are its
  if (t == T - 1) mine[A.cols - 1] += acc_edge;
  __syncthreads();
  for (int c = threadIdx.y * T + t; c < A.cols; c += T * blockDim.y) {
    float v = 0.0f;
    for (int y = 0; y < (int)blockDim.y; ++y) v += s_acc[(size_t)y * A.cols + c];
    A.partial[(int64_t)blockIdx.x * A.cols + c] = v;
  }
}

// Other rows that do not start on 16 bytes, through a ring of slots (as above).
// The gain of a thread's columns and its gradient stay in registers.  Bound by
// its instructions, which 15 to 20 warps per SM (for their registers) issue in
// two cycles of three.  9000 x 6001 fp32 with an odd stride: 165 us, 258 read
// twice by single elements; 6001 x 2049 bf16 with arrays that start unlike each
// other: 41 us, 54 by single elements in registers (in pairs in registers, where
// the arrays allow them, 26: hence the kernel above).  Four pairs per thread
// take 45 us, fewer registers (which spill) 49 and more.
constexpr int bwd_staged_threads = 512;

template <int DT, int V, bool DSUM>
__global__ void __launch_bounds__(bwd_staged_threads) rmsnorm_bwd_staged_kernel(const __grid_constant__ BwdArgs A, int stages) {
  using X = Pairs<DT, V>;
  constexpr int kArrays = DSUM ? 3 : 2;
  __shared__ float2 part[2][32];
  extern __shared__ __align__(16) unsigned char smem[];
  const int T = blockDim.x, t = threadIdx.x, bytes = slot_bytes(A.cols, elem_size(DT));
  depends_wait();
  unsigned char* ring = smem + (size_t)threadIdx.y * stages * kArrays * bytes;   // [stages][kArrays][bytes]
  float2 acc[V], gain[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int a = X::col(i, 0, t, T), b = X::col(i, 1, t, T);
    acc[i] = make_float2(0.0f, 0.0f);
    gain[i] = make_float2(a < A.cols ? A.gain[a] : 0.0f, b < A.cols ? A.gain[b] : 0.0f);
  }
  const Extent eh = extent_of<DT>(A.h, A.rows, A.ld_h, A.cols), ed = extent_of<DT>(A.dy, A.rows, A.ld_dy, A.cols),
               es = DSUM ? extent_of<DT>(A.dsum, A.rows, A.ld_dsum, A.cols) : eh;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const int64_t r0 = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const unsigned char *fh = row_of<DT>(A.h, r0, A.ld_h), *fd = row_of<DT>(A.dy, r0, A.ld_dy), *fs = row_of<DT>(A.dsum, r0, A.ld_dsum);
  const int64_t step_h = step * A.ld_h * elem_size(DT), step_d = step * A.ld_dy * elem_size(DT),
                step_s = step * A.ld_dsum * elem_size(DT), step_x = step * A.ld_dx * elem_size(DT);
  uint32_t oh = (uint32_t)(uintptr_t)fh, od = (uint32_t)(uintptr_t)fd, os = (uint32_t)(uintptr_t)fs;   // low bits of the computed row's
  int64_t ahead = r0;   // row that is fetched next
  auto issue = [&](unsigned char* slot) {
    if (ahead < A.rows) {
      stage_row<DT>(slot, eh, fh, A.cols, t, T);
      stage_row<DT>(slot + bytes, ed, fd, A.cols, t, T);
      if constexpr (DSUM) stage_row<DT>(slot + 2 * bytes, es, fs, A.cols, t, T);
    }
    async_commit();   // one group per row, empty past the end
    ahead += step;
    fh += step_h, fd += step_d, fs += step_s;
  };
  for (int s = 0; s < stages; ++s) issue(ring + s * kArrays * bytes);
  unsigned char* dx = row_of<DT>(A.dx, r0, A.ld_dx);
  int flip = 0, s = 0;
  // the same number of passes in every thread of the CTA
  for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < A.rows; base += step, flip ^= 1) {
    const bool live = base + threadIdx.y < A.rows;
    const int cols = live ? A.cols : 0;
    unsigned char* slot = ring + s * kArrays * bytes;
    wait_rows(stages - 1);
    row_sync<true>(T);   // the other threads' copies
    typename X::Raw rh[V], rd[V], rs[DSUM ? V : 1];
    X::load(slot, oh, cols, t, T, rh);
    X::load(slot + bytes, od, cols, t, T, rd);
    if constexpr (DSUM) X::load(slot + 2 * bytes, os, cols, t, T, rs);
    oh += (uint32_t)step_h, od += (uint32_t)step_d, os += (uint32_t)step_s;
    float2 sh = make_float2(0.0f, 0.0f), sa = sh;   // sums of h^2 and a h
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 h = X::unpack(rh[i]);
      sh = fma2(h, h, sh);
      sa = fma2(mul2_rn(X::unpack(rd[i]), gain[i]), h, sa);
    }
    const float2 sum = row_sum<true>(make_float2(sh.x + sh.y, sa.x + sa.y), T, part[flip]);
    if (T <= 32) __syncwarp();   // else row_sum's barrier: all threads of the row have read the slot
    issue(slot);
    const float inv = inverse_norm(sum.x, A.inv_cols, A.eps);
    const float c = -(sum.y * A.inv_cols * inv * inv);   // -mean(a h) inv^2
    if (live) {   // past the end inv is infinite where eps is zero
      float2 o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 h = X::unpack(rh[i]), d = X::unpack(rd[i]);
        const float2 e = fma2(h, make_float2(c, c), mul2_rn(d, gain[i]));
        if constexpr (DSUM) o[i] = fma2(e, make_float2(inv, inv), X::unpack(rs[i]));
        else o[i] = mul2_rn(e, inv);
        acc[i] = fma2(d, mul2_rn(h, inv), acc[i]);
      }
      X::store(dx, cols, t, T, o);
    }
    dx += step_x;
    s = s + 1 == stages ? 0 : s + 1;
  }
  float* out = A.partial + (int64_t)blockIdx.x * A.cols;
  float* mine = out;
  if (blockDim.y > 1) {
    async_wait<0>();
    __syncthreads();   // the ring is free
    mine = reinterpret_cast<float*>(smem) + (size_t)threadIdx.y * A.cols;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int a = X::col(i, 0, t, T), b = X::col(i, 1, t, T);
    if (a < A.cols) mine[a] = acc[i].x;
    if (b < A.cols) mine[b] = acc[i].y;
  }
  if (blockDim.y == 1) return;
  __syncthreads();
  for (int k = threadIdx.y * T + t; k < A.cols; k += T * blockDim.y) {
    float v = 0.0f;
    for (int y = 0; y < (int)blockDim.y; ++y) v += reinterpret_cast<const float*>(smem)[(size_t)y * A.cols + k];
    out[k] = v;
  }
}

// Longer rows: read twice.  A thread's columns are the same in every row; their
// sums lie in shared memory, or, where a row is too long for it, in the CTA's
// row of `partial`.  3005 x 11828 bf16 in pieces of 8 bytes: 65 us with three
// CTAs of 512 threads per SM, 86 with one of 1024.
constexpr int kWalkThreads = 512, kWalkPerSm = 3;

template <int DT, int N, bool IN_SMEM>
__global__ void __launch_bounds__(kWalkThreads, kWalkPerSm) rmsnorm_bwd_walk_kernel(const __grid_constant__ BwdArgs A) {
  __shared__ float2 part[2][32];
  extern __shared__ __align__(16) float s_acc[];
  const int T = blockDim.x, t = threadIdx.x;
  depends_wait();
  float* out = A.partial + (int64_t)blockIdx.x * A.cols;
  float* acc = IN_SMEM ? s_acc : out;
  for (int c = t * N; c < A.cols; c += T * N) {
    const float zero[N] = {};
    store_f32<N>(acc + c, zero);
  }
  int flip = 0;
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x, flip ^= 1) {
    const void* hp = row_of<DT>(A.h, row, A.ld_h);
    const void* dp = row_of<DT>(A.dy, row, A.ld_dy);
    float2 s = make_float2(0.0f, 0.0f);   // sums of h^2 and a h
#pragma unroll 4
    for (int c = t * N; c < A.cols; c += T * N) {
      float h[N], d[N], g[N];
      load_n<DT, N>(hp, c, h);
      load_n<DT, N>(dp, c, d);
      load_f32<N>(A.gain + c, g);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        s.x = fmaf(h[j], h[j], s.x);
        s.y = fmaf(d[j] * g[j], h[j], s.y);
      }
    }
    s = row_sum<false>(s, T, part[flip]);
    const float inv = inverse_norm(s.x, A.inv_cols, A.eps);
    const float k = s.y * A.inv_cols * inv * inv;
#pragma unroll 4
    for (int c = t * N; c < A.cols; c += T * N) {
      float h[N], d[N], g[N], o[N], sum[N];
      load_n<DT, N>(hp, c, h);
      load_n<DT, N>(dp, c, d);
      load_f32<N>(A.gain + c, g);
      load_f32<N>(acc + c, sum);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        o[j] = inv * (d[j] * g[j] - h[j] * k);
        sum[j] = fmaf(d[j], h[j] * inv, sum[j]);
      }
      store_f32<N>(acc + c, sum);
      if (A.dsum) {
        float f[N];
        load_n<DT, N>(row_of<DT>(A.dsum, row, A.ld_dsum), c, f);
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] += f[j];
      }
      store_n<DT, N>(row_of<DT>(A.dx, row, A.ld_dx), c, o);
    }
  }
  if constexpr (IN_SMEM) {
    for (int c = t * N; c < A.cols; c += T * N) {
      float sum[N];
      load_f32<N>(acc + c, sum);
      store_f32<N>(out + c, sum);
    }
  }
}

// dgain[c] = sum of n rows of partial, in an order that n alone fixes.  Bound by
// latency: two batches of loads and a reduction.
constexpr int kSlices = 32;

__global__ void __launch_bounds__(1024) dgain_kernel(const float* partial, int32_t n, int32_t cols, float* dgain) {
  __shared__ float s[kSlices][33];
  depends_wait();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.0f;
  if (c < cols) {
    const float* p = partial + c;
    constexpr int kAhead = 10;   // loads in flight
    for (int r = threadIdx.y; r < n; r += kAhead * kSlices) {
      float f[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) f[i] = r + i * kSlices < n ? __ldcg(p + (int64_t)(r + i * kSlices) * cols) : 0.0f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) v += f[i];
    }
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = s[threadIdx.x][threadIdx.y];   // a warp per column
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += lane_xor(v, o);
  const int cc = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && cc < cols) dgain[cc] = v;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool is_dtype(int v) { return v == QMUON_BF16 || v == QMUON_FP16 || v == QMUON_FP32; }

// Threads of a row and 16-byte vectors per thread: V is the largest up to
// `want` that leaves a row `least` threads, or the smallest that fits.  V == 0:
// none does.
struct Shape {
  int T, V;
  // rows of at most a warp: a CTA of 256 threads; of more: of `threads`, or one row
  dim3 block(int threads) const { return dim3(T, T <= 32 ? 256 / T : std::max(1, threads / T)); }
};

template <class MaxThreads>
Shape pick_shape(int nv, int want, int most, int least, MaxThreads max_threads) {
  int V = want;
  while (V > 1 && nv / V < least) V /= 2;
  for (; V <= most; V *= 2) {
    int T = (nv + V - 1) / V;
    if (T > 32) {
      T = (T + 31) / 32 * 32;
    } else {
      int p = least;
      while (p < T) p *= 2;
      T = p;
    }
    if (T <= max_threads(V)) return {T, V};
  }
  return {0, 0};
}

// Threads and pieces per thread of a row of n pieces: a warp with two or four for
// short rows (more would be tests without work: 300000 x 100 bf16 forward in
// 61 us with two, 91 with eight), else `want`, or eight where those need too
// many threads.  V == 0: too long.
Shape piece_shape(int n, int want, int max_threads) {
  if (n <= 64) return {32, 2};
  if (n <= 128) return {32, 4};
  for (int V = want; V <= 8; V *= 2) {
    const int T = ((n + V - 1) / V + 31) / 32 * 32;
    if (T <= max_threads) return {T, V};
  }
  return {0, 0};
}

int device_sms() {
  static std::atomic<int> cached[64] = {};
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if ((sms = cached[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  cached[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// CTAs of a kernel that an SM of the current device holds at once.  The first
// call for a kernel also lets it have kMaxSmem bytes of dynamic shared memory;
// later ones make no CUDA call but cudaGetDevice, so that they can be captured.
constexpr int kMaxSmem = 224 * 1024;
cudaError_t resident_ctas(const void* kernel, int threads, int smem, int* ctas) {
  static std::mutex mu;
  static std::map<std::tuple<const void*, int, int, int>, int> known;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  int& n = known[{kernel, dev, threads, smem}];
  if (n == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
    if (e != cudaSuccess) return e;
    n = std::max(n, 1);
  }
  *ctas = n;
  return cudaSuccess;
}

// Whether all rows of the arrays start alike within 4 bytes.
struct Strided {
  const void* p;
  int64_t ld;
};
bool rows_alike(std::initializer_list<Strided> arrays) {
  const Strided& a = *arrays.begin();
  for (const Strided& b : arrays)
    if (b.p && (((reinterpret_cast<uintptr_t>(a.p) ^ reinterpret_cast<uintptr_t>(b.p)) & 3) || ((a.ld ^ b.ld) & 1))) return false;
  return true;
}

template <int DT, bool RES, bool MX>
cudaError_t launch_fwd(const FwdArgs& A, cudaStream_t s) {
  constexpr int K = Vec16<DT>::kElems;
  // Four vectors per thread, so that a row takes few warps (and the bytes in flight are many); where rows do not fill
  // the SMs, one, so that a row is done sooner: one row of 4096 bf16 takes 3.7 us so,
  // 4.5 with four.
  const bool few = A.rows <= device_sms();
  const int least = MX && DT == QMUON_FP32 ? 8 : 4;   // the 32 elements of a scale lie in one access of a row's threads
  const Shape S = A.align == 16 ? pick_shape(A.cols / K, few ? 1 : 4, 4, least, fwd_max_threads) : Shape{0, 0};
  auto grid = [&](const dim3& b) { return (unsigned)std::min<int64_t>((A.rows + b.y - 1) / b.y, ((int64_t)1 << 31) - 1); };
  if (A.align == 16) {
    const dim3 block = S.V ? S.block(0) : dim3(1024);
    if (S.V == 1) return launch_dependent(rmsnorm_fwd_rows_kernel<DT, 1, RES, MX>, grid(block), block, 0, s, A);
    if (S.V == 2) return launch_dependent(rmsnorm_fwd_rows_kernel<DT, 2, RES, MX>, grid(block), block, 0, s, A);
    if (S.V == 4) return launch_dependent(rmsnorm_fwd_rows_kernel<DT, 4, RES, MX>, grid(block), block, 0, s, A);
    return launch_dependent(rmsnorm_fwd_walk_kernel<DT, K, MX>, grid(block), block, 0, s, A);
  }
  if constexpr (!MX) {
    // Pairs: four per thread (eight take 22.2 us for 6001 x 2049 fp16, four 20.6).  Single elements: eight; those of 16 bits
    // in rows of up to 128 columns only (300000 x 101 bf16 62 us, 84 by way of shared memory; 100000 x 257 57 and 49).
    const bool pairs = DT != QMUON_FP32 &&
                       rows_alike({{A.x, A.ld_x}, {A.residual, A.ld_residual}, {A.sum, A.ld_sum}, {A.y, A.ld_y}});
    const Shape C = piece_shape(A.cols / (pairs ? 2 : 1), pairs ? 4 : 8, 1024);
    const dim3 block = C.V ? C.block(0) : dim3(1);
    auto launch = [&](auto kernel) { return launch_dependent(kernel, grid(block), block, 0, s, A); };
    if constexpr (DT != QMUON_FP32) {
      if (pairs && C.V == 2) return launch(rmsnorm_fwd_pieces_kernel<DT, 2, 2, RES>);
      if (pairs && C.V == 4) return launch(rmsnorm_fwd_pieces_kernel<DT, 2, 4, RES>);
      if (pairs && C.V == 8) return launch(rmsnorm_fwd_pieces_kernel<DT, 2, 8, RES>);
    }
    if (!pairs && C.V == 2) return launch(rmsnorm_fwd_pieces_kernel<DT, 1, 2, RES>);
    if (!pairs && C.V == 4) return launch(rmsnorm_fwd_pieces_kernel<DT, 1, 4, RES>);
    if constexpr (DT == QMUON_FP32)
      if (C.V == 8) return launch(rmsnorm_fwd_pieces_kernel<DT, 1, 8, RES>);
  }
  if constexpr (MX || DT != QMUON_FP32) {
    // The 32 elements of a scale lie in one access of a row's threads.  Without a scale, rows that take more than 512
    // threads are as fast read twice (4000 x 12001 bf16 128 us, 136 so); with one, not (12032 columns 174 and 142).
    const Shape C = pick_shape((A.cols + 1) / 2, 8, 8, !MX ? 8 : DT == QMUON_FP32 ? 32 : 16, [](int) { return MX ? 1024 : 512; });
    if (C.V) {
      const dim3 block = C.block(0);
      const int smem = (RES ? 2 : 1) * (int)block.y * slot_bytes(A.cols, elem_size(DT));
      auto launch = [&](auto kernel) {
        int per_sm = 0;   // the query lets the kernel have its shared memory
        const cudaError_t e = resident_ctas(reinterpret_cast<const void*>(kernel), (int)(block.x * block.y), smem, &per_sm);
        return e != cudaSuccess ? e : launch_dependent(kernel, grid(block), block, smem, s, A);
      };
      if constexpr (MX) {   // the others have more than 128 columns: eight pairs
        if (C.V == 1) return launch(rmsnorm_fwd_staged_kernel<DT, 1, RES, MX>);
        if (C.V == 2) return launch(rmsnorm_fwd_staged_kernel<DT, 2, RES, MX>);
        if (C.V == 4) return launch(rmsnorm_fwd_staged_kernel<DT, 4, RES, MX>);
      }
      return launch(rmsnorm_fwd_staged_kernel<DT, 8, RES, MX>);
    }
  }
  const dim3 block(1024);
  if constexpr (!MX) {
    if (A.align == 8) return launch_dependent(rmsnorm_fwd_walk_kernel<DT, K / 2, MX>, grid(block), block, 0, s, A);
    if constexpr (K == 8)
      if (A.align == 4) return launch_dependent(rmsnorm_fwd_walk_kernel<DT, 2, MX>, grid(block), block, 0, s, A);
  }
  return launch_dependent(rmsnorm_fwd_walk_kernel<DT, 1, MX>, grid(block), block, 0, s, A);
}
template <int DT>
cudaError_t launch_fwd_dt(const FwdArgs& A, cudaStream_t s) {
  if (A.payload) return A.residual ? launch_fwd<DT, true, true>(A, s) : launch_fwd<DT, false, true>(A, s);
  return A.residual ? launch_fwd<DT, true, false>(A, s) : launch_fwd<DT, false, false>(A, s);
}

// CTAs of the backward pass, each with its row of `partial`: those that the SMs
// hold at once, at most four per SM.
constexpr int kBwdPerSm = 4;
int bwd_grid(int64_t groups, int sms, int per_sm) {
  return (int)std::min<int64_t>(std::max<int64_t>(groups, 1), (int64_t)sms * std::min(per_sm, kBwdPerSm));
}

template <class... Extra>
cudaError_t launch_bwd_kernel(void (*kernel)(BwdArgs, Extra...), const BwdArgs& A, dim3 block, int smem, int most, int sms,
                              int* grid, cudaStream_t s, Extra... extra) {
  int per_sm = 0;
  const cudaError_t e = resident_ctas(reinterpret_cast<const void*>(kernel), (int)(block.x * block.y), smem, &per_sm);
  if (e != cudaSuccess) return e;
  *grid = bwd_grid((A.rows + block.y - 1) / block.y, sms, std::min(per_sm, most));
  return launch_dependent(kernel, *grid, block, smem, s, A, extra...);
}

// `row`: bytes of a stage of the CTA's rings.
inline cudaError_t launch_bwd_ring(void (*kernel)(BwdArgs, int), const BwdArgs& A, const dim3& block, int row, int sms, int* grid,
                                   cudaStream_t s) {
  const int stages = std::min(3, std::max(1, kMaxSmem / row));
  const int smem = std::max(stages * row, block.y > 1 ? (int)block.y * A.cols * 4 : 0);
  // Rings of up to 150 KB per SM: more bytes in flight slow DRAM down.  16384 x 4096 bf16 takes 83 us with 147 KB (one
  // CTA of two rows), 91 with 221 (three of one row), 88 with 196 (four, two stages); 32768 x 1024 fp16 37 with 98, 39
  // with 196.
  return launch_bwd_kernel(kernel, A, block, smem, std::max(1, 150 * 1024 / smem), sms, grid, s, stages);
}
template <int DT, int V, bool DSUM>
cudaError_t launch_bwd_rows(const BwdArgs& A, const dim3& block, int sms, int* grid, cudaStream_t s) {
  return launch_bwd_ring(rmsnorm_bwd_rows_kernel<DT, V, DSUM>, A, block, (DSUM ? 3 : 2) * V * (int)(block.x * block.y) * 16, sms, grid,
                         s);
}

template <int DT, bool DSUM>
cudaError_t launch_bwd(const BwdArgs& A, int sms, int* grid, cudaStream_t s) {
  constexpr int K = Vec16<DT>::kElems;
  if (A.align == 16) {
    const Shape S = pick_shape(A.cols / K, 4, 8, 4, bwd_max_threads);
    // two or more rows per CTA, where there are enough of them
    const dim3 block = S.V ? S.block(A.rows >= 4 * (int64_t)sms ? 256 : 0) : dim3(1);
    if (S.V == 1) return launch_bwd_rows<DT, 1, DSUM>(A, block, sms, grid, s);
    if (S.V == 2) return launch_bwd_rows<DT, 2, DSUM>(A, block, sms, grid, s);
    if (S.V == 4) return launch_bwd_rows<DT, 4, DSUM>(A, block, sms, grid, s);
    if (S.V == 8) return launch_bwd_rows<DT, 8, DSUM>(A, block, sms, grid, s);
  } else {
    if constexpr (DT != QMUON_FP32) {
      const Shape C = piece_shape(A.cols / 2, 8, bwd_piece_threads);
      if (C.V && rows_alike({{A.h, A.ld_h}, {A.dy, A.ld_dy}, {A.dsum, A.ld_dsum}, {A.dx, A.ld_dx}})) {
        const dim3 block = C.block(256);
        const int smem = ((int)block.y * A.cols + C.T * C.V * 2 + 2) * 4;
        auto launch = [&](auto kernel) { return launch_bwd_kernel(kernel, A, block, smem, kBwdPerSm, sms, grid, s); };
        if (C.V == 2) return launch(rmsnorm_bwd_pieces_kernel<DT, 2, DSUM>);
        if (C.V == 4) return launch(rmsnorm_bwd_pieces_kernel<DT, 4, DSUM>);
        return launch(rmsnorm_bwd_pieces_kernel<DT, 8, DSUM>);
      }
    }
    const Shape C = pick_shape((A.cols + 1) / 2, 8, 8, 8, [](int) { return bwd_staged_threads; });
    if (C.V) {
      const dim3 block = C.block(256);
      const int row = (DSUM ? 3 : 2) * (int)block.y * slot_bytes(A.cols, elem_size(DT));
      auto launch = [&](auto kernel) { return launch_bwd_ring(kernel, A, block, row, sms, grid, s); };
      if (C.V == 1) return launch(rmsnorm_bwd_staged_kernel<DT, 1, DSUM>);
      if (C.V == 2) return launch(rmsnorm_bwd_staged_kernel<DT, 2, DSUM>);
      if (C.V == 4) return launch(rmsnorm_bwd_staged_kernel<DT, 4, DSUM>);
      return launch(rmsnorm_bwd_staged_kernel<DT, 8, DSUM>);
    }
  }
  const int64_t bytes = (int64_t)A.cols * 4;
  auto walk = [&](auto n) {
    constexpr int N = decltype(n)::value;
    return bytes <= kMaxSmem
               ? launch_bwd_kernel(rmsnorm_bwd_walk_kernel<DT, N, true>, A, kWalkThreads, (int)bytes, kBwdPerSm, sms, grid, s)
               : launch_bwd_kernel(rmsnorm_bwd_walk_kernel<DT, N, false>, A, kWalkThreads, 0, kBwdPerSm, sms, grid, s);
  };
  if (A.align == 16) return walk(std::integral_constant<int, K>{});
  if (A.align == 8) return walk(std::integral_constant<int, K / 2>{});
  if constexpr (K == 8)
    if (A.align == 4) return walk(std::integral_constant<int, 2>{});
  return walk(std::integral_constant<int, 1>{});
}
template <int DT>
cudaError_t launch_bwd_dt(const BwdArgs& A, int sms, int* grid, cudaStream_t s) {
  return A.dsum ? launch_bwd<DT, true>(A, sms, grid, s) : launch_bwd<DT, false>(A, sms, grid, s);
}

// A matrix argument: non-null, aligned to its elements, rows at least cols
// apart; `align` falls to the bytes on which its rows start.
bool check_matrix(const void* p, int64_t ld, int64_t cols, int dt, int* align) {
  const int es = elem_size(dt);
  if (!p || ld < cols || !is_aligned(p, es)) return false;
  while (!is_aligned(p, *align) || (ld * es) % *align) *align /= 2;
  return true;
}
// The bytes that a row's elements, its gain and an MXFP8 payload allow to move at once.
int row_align(int64_t cols, int dt, const float* gain, const uint8_t* payload) {
  const int es = elem_size(dt);
  int align = is_aligned(payload, 8) ? 16 : 8;
  while (align > es && ((cols * es) % align || !is_aligned(gain, std::min(16, 4 * align / es)))) align /= 2;
  return align;
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
  return no_throw("qmuon_rmsnorm_forward", [&]() -> qmuon_status {
    if (!n || !check_sizes(n->rows, n->cols, n->dtype, n->eps)) return QMUON_ERR_INVALID_ARGUMENT;
    if (n->rows == 0) return QMUON_OK;
    if ((!n->y && !n->payload) || (n->payload == nullptr) != (n->scale_inv == nullptr)) return QMUON_ERR_INVALID_ARGUMENT;
    if (n->payload && n->cols % QMUON_SCALE_BLOCK) return QMUON_ERR_UNSUPPORTED;
    int align = row_align(n->cols, n->dtype, n->gain, n->payload);
    if (!n->gain || !is_aligned(n->gain, 4) || !check_matrix(n->x, n->ld_x, n->cols, n->dtype, &align))
      return QMUON_ERR_INVALID_ARGUMENT;
    if (n->residual && !check_matrix(n->residual, n->ld_residual, n->cols, n->dtype, &align)) return QMUON_ERR_INVALID_ARGUMENT;
    if (n->sum && !check_matrix(n->sum, n->ld_sum, n->cols, n->dtype, &align)) return QMUON_ERR_INVALID_ARGUMENT;
    if (n->y && !check_matrix(n->y, n->ld_y, n->cols, n->dtype, &align)) return QMUON_ERR_INVALID_ARGUMENT;
    FwdArgs A{n->x,    n->residual,    n->gain,   n->sum,  n->y,    n->payload, n->scale_inv, n->rows,
              n->ld_x, n->ld_residual, n->ld_sum, n->ld_y, (int32_t)n->cols, align, n->eps, 1.0f / (float)n->cols};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = n->dtype == QMUON_BF16   ? launch_fwd_dt<QMUON_BF16>(A, s)
                          : n->dtype == QMUON_FP16 ? launch_fwd_dt<QMUON_FP16>(A, s)
                                                   : launch_fwd_dt<QMUON_FP32>(A, s);
    return e == cudaSuccess ? QMUON_OK : set_error("qmuon_rmsnorm_forward (launch)", e);
  });
}

extern "C" size_t qmuon_rmsnorm_workspace_size(int64_t rows, int64_t cols) {
  if (!check_sizes(rows, cols, QMUON_FP32, 0.0f)) return 0;
  const int sms = device_sms();
  return ((size_t)bwd_grid(rows, sms > 0 ? sms : 1, kBwdPerSm) * (size_t)cols * 4 + 255) / 256 * 256;
}

extern "C" qmuon_status qmuon_rmsnorm_backward(const qmuon_rmsnorm_grad* n, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("qmuon_rmsnorm_backward");
  return no_throw("qmuon_rmsnorm_backward", [&]() -> qmuon_status {
    if (!n || !check_sizes(n->rows, n->cols, n->dtype, n->eps)) return QMUON_ERR_INVALID_ARGUMENT;
    if (!n->dgain || !is_aligned(n->dgain, 4)) return QMUON_ERR_INVALID_ARGUMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n->rows == 0) {
      const cudaError_t e = cudaMemsetAsync(n->dgain, 0, (size_t)n->cols * 4, s);
      return e == cudaSuccess ? QMUON_OK : set_error("qmuon_rmsnorm_backward (memset)", e);
    }
    int align = row_align(n->cols, n->dtype, n->gain, nullptr);
    if (!n->gain || !is_aligned(n->gain, 4) || !ws || !is_aligned(ws, 256)) return QMUON_ERR_INVALID_ARGUMENT;
    if (!check_matrix(n->dy, n->ld_dy, n->cols, n->dtype, &align) || !check_matrix(n->h, n->ld_h, n->cols, n->dtype, &align) ||
        !check_matrix(n->dx, n->ld_dx, n->cols, n->dtype, &align))
      return QMUON_ERR_INVALID_ARGUMENT;
    if (n->dsum && !check_matrix(n->dsum, n->ld_dsum, n->cols, n->dtype, &align)) return QMUON_ERR_INVALID_ARGUMENT;
    const int sms = device_sms();
    if (sms <= 0) return set_error_msg("qmuon_rmsnorm_backward: SM count query failed", QMUON_ERR_CUDA);
    if (ws_bytes < qmuon_rmsnorm_workspace_size(n->rows, n->cols)) return QMUON_ERR_WORKSPACE_TOO_SMALL;
    BwdArgs A{n->dy,    n->h,    n->dsum,    n->gain,  n->dx,            static_cast<float*>(ws), n->rows,
              n->ld_dy, n->ld_h, n->ld_dsum, n->ld_dx, (int32_t)n->cols, align, n->eps, 1.0f / (float)n->cols};
    int grid = 0;
    cudaError_t e = n->dtype == QMUON_BF16   ? launch_bwd_dt<QMUON_BF16>(A, sms, &grid, s)
                    : n->dtype == QMUON_FP16 ? launch_bwd_dt<QMUON_FP16>(A, sms, &grid, s)
                                             : launch_bwd_dt<QMUON_FP32>(A, sms, &grid, s);
    if (e == cudaSuccess)
      e = launch_dependent(dgain_kernel, (unsigned)((n->cols + 31) / 32), dim3(32, kSlices), 0, s, A.partial, grid, A.cols,
                           n->dgain);
    return e == cudaSuccess ? QMUON_OK : set_error("qmuon_rmsnorm_backward (launch)", e);
  });
}
