// Global gradient clipping and the AdamW step over many tensors.
//
// Both walk a list of tensors of any sizes cut into chunks: a plan's device
// table says which tensor each chunk belongs to, and one CTA takes one chunk
// (or, in the norm, every gridDim.x-th one).  There is no work per tensor, so
// hundreds of short vectors cost what one tensor of their total size costs.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <memory>
#include <vector>

#include "qm_elem.h"

namespace qm {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxElems = (int64_t)1 << 40;   // elements of one tensor

// ---------------------------------------------------------------------------
// global norm and clipping
// ---------------------------------------------------------------------------
constexpr int kClipChunk = 8192;   // elements

struct ClipTensor {
  void* grad;
  int64_t numel;
  int32_t first_chunk;
  int16_t dtype;
  int16_t vec;         // 16-byte aligned
};

struct ClipLaunch {
  const ClipTensor* tensors;
  const int32_t* chunk_tensor;
  int32_t n_chunks;
  unsigned int* ticket;   // the plan's: 0 between calls
  double* partials;       // workspace, one per CTA
  float* norm;            // [2]: norm, coefficient
  float max_norm;
};

template <int DT>
__device__ __forceinline__ float chunk_sumsq(const ClipTensor& T, int64_t e0, int n, int tid) {
  constexpr int K = Vec16<DT>::kElems;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  int done = 0;
  const unsigned char* base = static_cast<const unsigned char*>(T.grad) + e0 * elem_size(DT);
  if (T.vec) {
    const uint4* p = reinterpret_cast<const uint4*>(base);
    const int nv = n / K;
#pragma unroll 4
    for (int i = tid; i < nv; i += kThreads) {
      float f[K];
      Vec16<DT>::unpack(__ldg(p + i), f);
#pragma unroll
      for (int j = 0; j < K; ++j) s[j & 3] = fmaf(f[j], f[j], s[j & 3]);
    }
    done = nv * K;
  }
  for (int i = done + tid; i < n; i += kThreads) {
    const float f = load_elem<DT>(base, i);
    s[0] = fmaf(f, f, s[0]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__global__ void __launch_bounds__(kThreads) clip_norm_kernel(const ClipLaunch L) {
  __shared__ double s_warp[kThreads / 32];
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  double acc = 0.0;
  for (int c = blockIdx.x; c < L.n_chunks; c += gridDim.x) {
    const ClipTensor T = L.tensors[__ldg(L.chunk_tensor + c)];
    const int64_t e0 = (int64_t)(c - T.first_chunk) * kClipChunk;
    const int n = (int)min(T.numel - e0, (int64_t)kClipChunk);
    const float s = T.dtype == QMUON_BF16   ? chunk_sumsq<QMUON_BF16>(T, e0, n, tid)
                    : T.dtype == QMUON_FP16 ? chunk_sumsq<QMUON_FP16>(T, e0, n, tid)
                                            : chunk_sumsq<QMUON_FP32>(T, e0, n, tid);
    acc += (double)s;
  }
  auto block_sum = [&](double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) s_warp[warp] = v;
    __syncthreads();
    double t = 0.0;
    if (tid == 0)
      for (int w = 0; w < kThreads / 32; ++w) t += s_warp[w];
    return t;   // thread 0's
  };
  const double mine = block_sum(acc);
  if (tid == 0) {
    L.partials[blockIdx.x] = mine;
    __threadfence();
    s_last = atomicAdd(L.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  // the CTA that comes last adds the partial sums in CTA order
  __threadfence();
  double t = 0.0;
  for (int i = tid; i < (int)gridDim.x; i += kThreads) t += __ldcg(L.partials + i);
  const double total = block_sum(t);
  if (tid == 0) {
    const float norm = (float)sqrt(total);
    L.norm[0] = norm;
    // not finite: no coefficient, and whatever takes it leaves its tensors alone
    L.norm[1] = isfinite(norm) ? fminf(1.0f, __fdiv_rn(L.max_norm, __fadd_rn(norm, 1e-6f))) : __int_as_float(0x7FC00000);
    *L.ticket = 0u;
  }
}

template <int DT>
__device__ __forceinline__ void chunk_scale(const ClipTensor& T, int64_t e0, int n, int tid, float c) {
  constexpr int K = Vec16<DT>::kElems;
  int done = 0;
  unsigned char* base = static_cast<unsigned char*>(T.grad) + e0 * elem_size(DT);
  if (T.vec) {
    uint4* p = reinterpret_cast<uint4*>(base);
    const int nv = n / K;
#pragma unroll 4
    for (int i = tid; i < nv; i += kThreads) {
      float f[K];
      Vec16<DT>::unpack(p[i], f);
#pragma unroll
      for (int j = 0; j < K; ++j) f[j] *= c;
      p[i] = Vec16<DT>::pack(f);
    }
    done = nv * K;
  }
  for (int i = done + tid; i < n; i += kThreads) store_elem<DT>(base, i, load_elem<DT>(base, i) * c);
}

__global__ void __launch_bounds__(kThreads) clip_scale_kernel(const ClipLaunch L) {
  const float c = __ldg(L.norm + 1);
  if (!(c < 1.0f)) return;   // within the bound, or not finite
  const int k = blockIdx.x;
  const ClipTensor T = L.tensors[__ldg(L.chunk_tensor + k)];
  const int64_t e0 = (int64_t)(k - T.first_chunk) * kClipChunk;
  const int n = (int)min(T.numel - e0, (int64_t)kClipChunk);
  if (T.dtype == QMUON_BF16) chunk_scale<QMUON_BF16>(T, e0, n, threadIdx.x, c);
  else if (T.dtype == QMUON_FP16) chunk_scale<QMUON_FP16>(T, e0, n, threadIdx.x, c);
  else chunk_scale<QMUON_FP32>(T, e0, n, threadIdx.x, c);
}

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------
// With g' = c g (c the clipping coefficient), every operation rounded once:
//   m <- b1 m + (1 - b1) g'          v <- b2 v + (1 - b2) g'^2
//   p <- p (1 - lr wd) - (lr / (1 - b1^t)) (m / (sqrt(v) / sqrt(1 - b2^t) + eps))
constexpr int kAdamChunk = 2048;   // elements: 8 per thread, or one 256-element block per warp

struct AdamTensor {
  float* param;
  const void* grad;
  void* copy;          // 16-bit copy of the parameters, or null
  void* m;
  void* v;
  float* m_absmax;     // 8-bit states
  float* v_absmax;
  int64_t numel;
  float lr_scale, weight_decay;
  int32_t first_chunk;
  int32_t index;       // in the caller's list: the stochastic rounding's counter
  int16_t grad_dtype, copy_dtype;
  int16_t vec;         // four elements of every array can be moved at once
  int16_t pad;
};

struct AdamLaunch {
  const AdamTensor* tensors;
  const int32_t* chunk_tensor;
  const float* grad_scale;   // D, or null
  float lr, b1, omb1, b2, omb2, rbc1, rbc2, eps;
  uint32_t key0, key1, step;
};

struct AdamCoef {
  float scale, decay, step;
};

__device__ __forceinline__ AdamCoef adam_coef(const AdamLaunch& L, const AdamTensor& T, float scale) {
  const float lr = __fmul_rn(L.lr, T.lr_scale);
  return {scale, __fsub_rn(1.0f, __fmul_rn(lr, T.weight_decay)), __fmul_rn(lr, L.rbc1)};
}

// New momentum, second moment and parameter of one element; returns sqrt(v).
__device__ __forceinline__ float adam_elem(const AdamLaunch& L, const AdamCoef& C, float g, float& p, float& m, float& v) {
  g = __fmul_rn(g, C.scale);
  m = __fadd_rn(__fmul_rn(m, L.b1), __fmul_rn(g, L.omb1));
  v = __fadd_rn(__fmul_rn(v, L.b2), __fmul_rn(__fmul_rn(g, g), L.omb2));
  const float r = __fsqrt_rn(v);
  const float u = __fdiv_rn(m, __fadd_rn(__fmul_rn(r, L.rbc2), L.eps));
  p = __fsub_rn(__fmul_rn(p, C.decay), __fmul_rn(C.step, u));
  return r;
}

// Four elements from e, of which the first n exist.
__device__ __forceinline__ void load4(const float* p, int64_t e, int n, bool vec, float* f) {
  if (vec && n == 4) {
    const float4 t = __ldcs(reinterpret_cast<const float4*>(p + e));
    f[0] = t.x, f[1] = t.y, f[2] = t.z, f[3] = t.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = j < n ? p[e + j] : 0.0f;
  }
}
__device__ __forceinline__ void store4(float* p, int64_t e, int n, bool vec, const float* f) {
  if (vec && n == 4) {
    __stcs(reinterpret_cast<float4*>(p + e), make_float4(f[0], f[1], f[2], f[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) p[e + j] = f[j];
  }
}
template <int DT>
__device__ __forceinline__ void load4_16(const void* p, int64_t e, int n, bool vec, float* f) {
  if (vec && n == 4) {
    const uint2 t = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + e));
    const float2 a = unpack2<DT>(t.x), b = unpack2<DT>(t.y);
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = j < n ? load_elem<DT>(p, e + j) : 0.0f;
  }
}
__device__ __forceinline__ void load_grad4(const AdamTensor& T, int64_t e, int n, float* f) {
  if (T.grad_dtype == QMUON_FP32) load4(static_cast<const float*>(T.grad), e, n, T.vec, f);
  else if (T.grad_dtype == QMUON_BF16) load4_16<QMUON_BF16>(T.grad, e, n, T.vec, f);
  else load4_16<QMUON_FP16>(T.grad, e, n, T.vec, f);
}
template <int DT>
__device__ __forceinline__ void store4_16(void* p, int64_t e, int n, bool vec, const float* f) {
  if (vec && n == 4) {
    __stcs(reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + e),
           make_uint2(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3])));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) store_elem<DT>(p, e + j, f[j]);
  }
}
__device__ __forceinline__ void store_copy4(const AdamTensor& T, int64_t e, int n, const float* f) {
  if (!T.copy) return;
  if (T.copy_dtype == QMUON_BF16) store4_16<QMUON_BF16>(T.copy, e, n, T.vec, f);
  else store4_16<QMUON_FP16>(T.copy, e, n, T.vec, f);
}

__global__ void __launch_bounds__(kThreads) adamw_f32_kernel(const __grid_constant__ AdamLaunch L) {
  const float scale = L.grad_scale ? __ldg(L.grad_scale) : 1.0f;
  if (!isfinite(scale)) return;
  const AdamTensor T = L.tensors[__ldg(L.chunk_tensor + blockIdx.x)];
  const AdamCoef C = adam_coef(L, T, scale);
  const int64_t e0 = (int64_t)((int)blockIdx.x - T.first_chunk) * kAdamChunk + threadIdx.x * 4;
  float p[2][4], m[2][4], v[2][4], g[2][4];
  int n[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t e = e0 + k * kThreads * 4;
    n[k] = (int)max((int64_t)0, min((int64_t)4, T.numel - e));
    load_grad4(T, e, n[k], g[k]);
    load4(T.param, e, n[k], T.vec, p[k]);
    load4(static_cast<const float*>(T.m), e, n[k], T.vec, m[k]);
    load4(static_cast<const float*>(T.v), e, n[k], T.vec, v[k]);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t e = e0 + k * kThreads * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) adam_elem(L, C, g[k][j], p[k][j], m[k][j], v[k][j]);
    store4(T.param, e, n[k], T.vec, p[k]);
    store4(static_cast<float*>(T.m), e, n[k], T.vec, m[k]);
    store4(static_cast<float*>(T.v), e, n[k], T.vec, v[k]);
    store_copy4(T, e, n[k], p[k]);
  }
}

// 8-bit states.  m and r = sqrt(v) are E4M3 codes with one fp32 maximum per
// 256 elements: x = code * (max / 448).  The root is stored, not v: its codes
// then cover as many powers of two as the momentum's, so that where r rounds
// to zero m does too, and no element divides a momentum by eps alone.
//
// A warp takes a block: lane l holds elements 4l..4l+3 and 128+4l..128+4l+3,
// so every load and store of the warp is one contiguous run.
__device__ __forceinline__ uint32_t load_codes4(const uint8_t* p, int64_t e, int n) {
  if (n == 4) return __ldcs(reinterpret_cast<const uint32_t*>(p + e));   // block starts are 16-byte aligned
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < n) w |= (uint32_t)p[e + j] << (8 * j);
  return w;
}
__device__ __forceinline__ void store_codes4(uint8_t* p, int64_t e, int n, uint32_t w) {
  if (n == 4) {
    __stcs(reinterpret_cast<uint32_t*>(p + e), w);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) p[e + j] = (uint8_t)(w >> (8 * j));
  }
}
__device__ __forceinline__ uint32_t encode4(const float* x, float sc) {
  return e4m3x2_of(__fmul_rn(x[0], sc), __fmul_rn(x[1], sc)) |
         (e4m3x2_of(__fmul_rn(x[2], sc), __fmul_rn(x[3], sc)) << 16);
}
// E4M3 of x with 16 random bits u: rounded up in magnitude with probability
// (remainder / step) to 2^-16.  2^-120 |x| has its exponent field where the
// code's is, subnormals included, so the bits above the lowest 20 are the code.
__device__ __forceinline__ uint32_t encode_sr(float x, uint32_t u) {
  const uint32_t b = __float_as_uint(__fmul_rn(fabsf(x), 7.52316384526264e-37f));
  const uint32_t c = min((b + (u << 4)) >> 20, 0x7Eu) | ((__float_as_uint(x) >> 24) & 0x80u);
  return x != x ? 0x7Fu : c;
}

template <bool SR>
__global__ void __launch_bounds__(kThreads) adamw_e4m3_kernel(const __grid_constant__ AdamLaunch L) {
  const float scale = L.grad_scale ? __ldg(L.grad_scale) : 1.0f;
  if (!isfinite(scale)) return;
  const AdamTensor T = L.tensors[__ldg(L.chunk_tensor + blockIdx.x)];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t blk = (int64_t)((int)blockIdx.x - T.first_chunk) * (kAdamChunk / kBlock) + warp;
  const int64_t b0 = blk * kBlock;
  if (b0 >= T.numel) return;   // the whole warp
  const AdamCoef C = adam_coef(L, T, scale);
  float p[2][4], m[2][4], v[2][4], g[2][4];
  uint32_t mc[2], vc[2];
  int n[2];
  const float m_unit = __fdiv_rn(T.m_absmax[blk], 448.0f), r_unit = __fdiv_rn(T.v_absmax[blk], 448.0f);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t e = b0 + k * 128 + lane * 4;
    n[k] = (int)max((int64_t)0, min((int64_t)4, T.numel - e));
    load_grad4(T, e, n[k], g[k]);
    load4(T.param, e, n[k], T.vec, p[k]);
    mc[k] = load_codes4(static_cast<const uint8_t*>(T.m), e, n[k]);
    vc[k] = load_codes4(static_cast<const uint8_t*>(T.v), e, n[k]);
  }
  float m_max = 0.0f, r_max = 0.0f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float2 ma = e4m3x2_to(mc[k]), mb = e4m3x2_to(mc[k] >> 16), va = e4m3x2_to(vc[k]), vb = e4m3x2_to(vc[k] >> 16);
    const float mo[4] = {ma.x, ma.y, mb.x, mb.y}, ro[4] = {va.x, va.y, vb.x, vb.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[k][j] = __fmul_rn(mo[j], m_unit);
      const float r = __fmul_rn(ro[j], r_unit);
      v[k][j] = __fmul_rn(r, r);
      v[k][j] = adam_elem(L, C, g[k][j], p[k][j], m[k][j], v[k][j]);   // the root from here on
      if (j >= n[k]) m[k][j] = v[k][j] = 0.0f;
      m_max = fmaxf(m_max, fabsf(m[k][j]));
      r_max = fmaxf(r_max, v[k][j]);
    }
  }
  m_max = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m_max)));   // not negative: ordered as integers
  r_max = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(r_max)));
  constexpr float kMax = 3.402823466e+38f;   // a zero or tiny maximum: no infinite factor
  const float m_sc = fminf(__fdiv_rn(448.0f, m_max), kMax), r_sc = fminf(__fdiv_rn(448.0f, r_max), kMax);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t e = b0 + k * 128 + lane * 4;
    uint32_t mo, vo;
    if constexpr (SR) {
      const uint64_t j = (uint64_t)e >> 2;
      const uint4 w = philox(make_uint4((uint32_t)j, (uint32_t)(j >> 32), (uint32_t)T.index, L.step), L.key0, L.key1);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      mo = vo = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mo |= encode_sr(__fmul_rn(m[k][i], m_sc), u[i] & 0xFFFFu) << (8 * i);
        vo |= encode_sr(__fmul_rn(v[k][i], r_sc), u[i] >> 16) << (8 * i);
      }
    } else {
      mo = encode4(m[k], m_sc);
      vo = encode4(v[k], r_sc);
    }
    store_codes4(static_cast<uint8_t*>(T.m), e, n[k], mo);
    store_codes4(static_cast<uint8_t*>(T.v), e, n[k], vo);
    store4(T.param, e, n[k], T.vec, p[k]);
    store_copy4(T, e, n[k], p[k]);
  }
  if (lane == 0) {
    T.m_absmax[blk] = m_max;
    T.v_absmax[blk] = r_max;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool is_dtype(int v) { return v == QMUON_BF16 || v == QMUON_FP16 || v == QMUON_FP32; }

// The chunks' table: for each chunk of `chunk` elements, the position of its
// tensor among the non-empty ones.
struct Chunks {
  std::vector<int32_t> tensor;
  std::vector<int32_t> first;   // per non-empty tensor
  bool add(int64_t numel, int64_t chunk) {
    const int64_t k = (numel + chunk - 1) / chunk;
    if ((int64_t)tensor.size() + k > ((int64_t)1 << 31) - 1) return false;
    first.push_back((int32_t)tensor.size());
    tensor.insert(tensor.end(), (size_t)k, (int32_t)first.size() - 1);
    return true;
  }
};

// One device allocation holding [head bytes, zeroed | tensors | chunk table].
template <class Tensor>
cudaError_t upload(const std::vector<Tensor>& ts, const std::vector<int32_t>& chunks, void** table, Tensor** d_ts,
                   int32_t** d_chunks) {
  constexpr size_t head = 256;
  const size_t tb = (ts.size() * sizeof(Tensor) + 255) / 256 * 256;
  std::vector<unsigned char> blob(head + tb + chunks.size() * 4, 0);
  std::memcpy(blob.data() + head, ts.data(), ts.size() * sizeof(Tensor));
  std::memcpy(blob.data() + head + tb, chunks.data(), chunks.size() * 4);
  cudaError_t e = cudaMalloc(table, blob.size());
  if (e != cudaSuccess) return e;
  e = cudaMemcpy(*table, blob.data(), blob.size(), cudaMemcpyHostToDevice);
  if (e != cudaSuccess) {
    cudaFree(*table);
    *table = nullptr;
    return e;
  }
  unsigned char* b = static_cast<unsigned char*>(*table);
  *d_ts = reinterpret_cast<Tensor*>(b + head);
  *d_chunks = reinterpret_cast<int32_t*>(b + head + tb);
  return cudaSuccess;
}

}  // namespace
}  // namespace qm

using namespace qm;

struct qmuon_clip_plan {
  void* table = nullptr;   // the ticket is its first word
  ClipTensor* tensors = nullptr;
  int32_t* chunk_tensor = nullptr;
  int32_t n_chunks = 0;
  int32_t grid = 0;
};

struct qmuon_adamw_plan {
  void* table = nullptr;
  AdamTensor* tensors = nullptr;
  int32_t* chunk_tensor = nullptr;
  int32_t n_chunks = 0;
  qmuon_state_kind state = QMUON_STATE_F32;
};

extern "C" qmuon_status qmuon_clip_plan_create(const qmuon_grad* grads, int32_t n, qmuon_clip_plan** out) {
  NvtxRange nvtx_range("qmuon_clip_plan_create");
  return no_throw("qmuon_clip_plan_create", [&]() -> qmuon_status {
    if (!out) return QMUON_ERR_INVALID_ARGUMENT;
    *out = nullptr;
    if (!grads || n <= 0) return QMUON_ERR_INVALID_ARGUMENT;
    Chunks ch;
    std::vector<ClipTensor> ts;
    for (int32_t i = 0; i < n; ++i) {
      const qmuon_grad& g = grads[i];
      if (!is_dtype(g.dtype) || g.numel < 0 || g.numel > kMaxElems) return QMUON_ERR_INVALID_ARGUMENT;
      if (g.numel == 0) continue;
      if (!g.grad || !is_aligned(g.grad, elem_size(g.dtype))) return QMUON_ERR_INVALID_ARGUMENT;
      if (!ch.add(g.numel, kClipChunk)) return QMUON_ERR_INVALID_ARGUMENT;
      ts.push_back({g.grad, g.numel, ch.first.back(), (int16_t)g.dtype, (int16_t)is_aligned(g.grad, 16)});
    }
    if (ts.empty()) return QMUON_ERR_INVALID_ARGUMENT;
    std::unique_ptr<qmuon_clip_plan> P(new qmuon_clip_plan);
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, clip_norm_kernel, kThreads, 0);
    if (e != cudaSuccess) return set_error("qmuon_clip_plan_create (device)", e);
    P->n_chunks = (int32_t)ch.tensor.size();
    P->grid = std::min(P->n_chunks, sms * std::max(per_sm, 1));
    e = upload(ts, ch.tensor, &P->table, &P->tensors, &P->chunk_tensor);
    if (e != cudaSuccess) return set_error("qmuon_clip_plan_create (tables)", e);
    *out = P.release();
    return QMUON_OK;
  });
}

extern "C" void qmuon_clip_plan_destroy(qmuon_clip_plan* plan) {
  if (!plan) return;
  cudaFree(plan->table);
  delete plan;
}

extern "C" size_t qmuon_clip_workspace_size(const qmuon_clip_plan* plan) {
  return plan ? ((size_t)plan->grid * sizeof(double) + 255) / 256 * 256 : 0;
}

extern "C" qmuon_status qmuon_grad_clip(const qmuon_clip_plan* plan, float max_norm, int32_t apply, float* norm, void* ws,
                                        size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("qmuon_grad_clip");
  if (!plan || !norm || !ws || !is_aligned(norm, 4) || !is_aligned(ws, 256)) return QMUON_ERR_INVALID_ARGUMENT;
  if (!(max_norm > 0.0f) || (apply != 0 && apply != 1)) return QMUON_ERR_INVALID_ARGUMENT;
  if (ws_bytes < qmuon_clip_workspace_size(plan)) return QMUON_ERR_WORKSPACE_TOO_SMALL;
  ClipLaunch L{};
  L.tensors = plan->tensors;
  L.chunk_tensor = plan->chunk_tensor;
  L.n_chunks = plan->n_chunks;
  L.ticket = static_cast<unsigned int*>(plan->table);
  L.partials = static_cast<double*>(ws);
  L.norm = norm;
  L.max_norm = max_norm;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  clip_norm_kernel<<<plan->grid, kThreads, 0, s>>>(L);
  if (apply) clip_scale_kernel<<<plan->n_chunks, kThreads, 0, s>>>(L);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? QMUON_OK : set_error("qmuon_grad_clip (launch)", e);
}

extern "C" qmuon_status qmuon_adamw_plan_create(const qmuon_adamw_tensor* tensors, int32_t n, qmuon_state_kind state,
                                                qmuon_adamw_plan** out) {
  NvtxRange nvtx_range("qmuon_adamw_plan_create");
  return no_throw("qmuon_adamw_plan_create", [&]() -> qmuon_status {
    if (!out) return QMUON_ERR_INVALID_ARGUMENT;
    *out = nullptr;
    if (!tensors || n <= 0 || (state != QMUON_STATE_F32 && state != QMUON_STATE_E4M3)) return QMUON_ERR_INVALID_ARGUMENT;
    const bool f32 = state == QMUON_STATE_F32;
    Chunks ch;
    std::vector<AdamTensor> ts;
    for (int32_t i = 0; i < n; ++i) {
      const qmuon_adamw_tensor& t = tensors[i];
      if (!is_dtype(t.grad_dtype) || t.numel < 0 || t.numel > kMaxElems) return QMUON_ERR_INVALID_ARGUMENT;
      if (!std::isfinite(t.lr_scale) || !std::isfinite(t.weight_decay)) return QMUON_ERR_INVALID_ARGUMENT;
      if (t.copy && t.copy_dtype != QMUON_BF16 && t.copy_dtype != QMUON_FP16) return QMUON_ERR_INVALID_ARGUMENT;
      if (t.numel == 0) continue;
      const size_t gs = elem_size(t.grad_dtype);
      if (!t.param || !t.grad || !t.m || !t.v) return QMUON_ERR_INVALID_ARGUMENT;
      if (!is_aligned(t.param, 4) || !is_aligned(t.grad, gs) || !is_aligned(t.copy, 2)) return QMUON_ERR_INVALID_ARGUMENT;
      if (!is_aligned(t.m, f32 ? 4 : 16) || !is_aligned(t.v, f32 ? 4 : 16)) return QMUON_ERR_INVALID_ARGUMENT;
      if (!f32 && (!t.m_absmax || !t.v_absmax || !is_aligned(t.m_absmax, 4) || !is_aligned(t.v_absmax, 4)))
        return QMUON_ERR_INVALID_ARGUMENT;
      if (!ch.add(t.numel, kAdamChunk)) return QMUON_ERR_INVALID_ARGUMENT;
      AdamTensor a{};
      a.param = t.param;
      a.grad = t.grad;
      a.copy = t.copy;
      a.m = t.m;
      a.v = t.v;
      a.m_absmax = t.m_absmax;
      a.v_absmax = t.v_absmax;
      a.numel = t.numel;
      a.lr_scale = t.lr_scale;
      a.weight_decay = t.weight_decay;
      a.first_chunk = ch.first.back();
      a.index = i;
      a.grad_dtype = (int16_t)t.grad_dtype;
      a.copy_dtype = (int16_t)t.copy_dtype;
      a.vec = is_aligned(t.param, 16) && is_aligned(t.grad, 4 * gs) && is_aligned(t.copy, 8) && is_aligned(t.m, 16) &&
              is_aligned(t.v, 16);
      ts.push_back(a);
    }
    if (ts.empty()) return QMUON_ERR_INVALID_ARGUMENT;
    std::unique_ptr<qmuon_adamw_plan> P(new qmuon_adamw_plan);
    P->state = state;
    P->n_chunks = (int32_t)ch.tensor.size();
    const cudaError_t e = upload(ts, ch.tensor, &P->table, &P->tensors, &P->chunk_tensor);
    if (e != cudaSuccess) return set_error("qmuon_adamw_plan_create (tables)", e);
    *out = P.release();
    return QMUON_OK;
  });
}

extern "C" void qmuon_adamw_plan_destroy(qmuon_adamw_plan* plan) {
  if (!plan) return;
  cudaFree(plan->table);
  delete plan;
}

namespace {

qmuon_status adamw_step(const char* where, const qmuon_adamw_plan* plan, int64_t t, double lr, double beta1, double beta2,
                        double eps, bool sr, uint64_t seed, const float* grad_scale, void* stream) {
  if (!plan || t < 1 || !is_aligned(grad_scale, 4)) return QMUON_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(lr) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0))
    return QMUON_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(eps) || !((float)eps > 0.0f)) return QMUON_ERR_INVALID_ARGUMENT;
  if (sr && plan->state != QMUON_STATE_E4M3) return QMUON_ERR_UNSUPPORTED;
  AdamLaunch L{};
  L.tensors = plan->tensors;
  L.chunk_tensor = plan->chunk_tensor;
  L.grad_scale = grad_scale;
  L.lr = (float)lr;
  L.b1 = (float)beta1;
  L.omb1 = (float)(1.0 - beta1);
  L.b2 = (float)beta2;
  L.omb2 = (float)(1.0 - beta2);
  L.rbc1 = (float)(1.0 / (1.0 - std::pow(beta1, (double)t)));
  L.rbc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)t)));
  L.eps = (float)eps;
  L.key0 = (uint32_t)seed;
  L.key1 = (uint32_t)(seed >> 32);
  L.step = (uint32_t)t;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (plan->state == QMUON_STATE_F32) adamw_f32_kernel<<<plan->n_chunks, kThreads, 0, s>>>(L);
  else if (sr) adamw_e4m3_kernel<true><<<plan->n_chunks, kThreads, 0, s>>>(L);
  else adamw_e4m3_kernel<false><<<plan->n_chunks, kThreads, 0, s>>>(L);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? QMUON_OK : set_error(where, e);
}

}  // namespace

extern "C" qmuon_status qmuon_adamw_step(const qmuon_adamw_plan* plan, int64_t t, double lr, double beta1, double beta2,
                                         double eps, const float* grad_scale, void* stream) {
  NvtxRange nvtx_range("qmuon_adamw_step");
  return adamw_step("qmuon_adamw_step (launch)", plan, t, lr, beta1, beta2, eps, false, 0, grad_scale, stream);
}

extern "C" qmuon_status qmuon_adamw_step_sr(const qmuon_adamw_plan* plan, int64_t t, double lr, double beta1, double beta2,
                                            double eps, uint64_t seed, const float* grad_scale, void* stream) {
  NvtxRange nvtx_range("qmuon_adamw_step_sr");
  return adamw_step("qmuon_adamw_step_sr (launch)", plan, t, lr, beta1, beta2, eps, true, seed, grad_scale, stream);
}
