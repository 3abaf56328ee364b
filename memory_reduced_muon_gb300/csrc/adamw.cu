// Global gradient clipping and the AdamW step over many tensors.
//
// Both walk a list of tensors of any sizes cut into chunks, of which a plan
// keeps a device table; one CTA takes one chunk (or, in the norm, every
// gridDim.x-th one).  There is no work per tensor, so hundreds of short vectors
// cost what one tensor of their total size costs.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <memory>
#include <type_traits>
#include <vector>

#include "qm_elem.h"

namespace qm {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxElems = (int64_t)1 << 40;         // elements of one tensor
constexpr int64_t kMaxChunks = (int64_t)1 << 30;        // of a plan: a grid's CTAs, and int indexes beyond them

// ---------------------------------------------------------------------------
// global norm and clipping
// ---------------------------------------------------------------------------
constexpr int kClipChunk = 8192;   // elements

struct ClipChunk {
  void* grad;
  int32_t n;           // elements, up to kClipChunk
  int16_t dtype;
  int16_t vec;         // 16-byte aligned
};

struct ClipLaunch {
  const ClipChunk* chunks;
  int32_t n_chunks;
  unsigned int* ticket;   // the plan's: 0 between calls
  double* partials;       // workspace, one per CTA
  float* norm;            // [2]: norm, coefficient
  float max_norm;
};

// A thread's share of a chunk, up to 32 squares, in four running sums: a sum's
// error grows with its additions, of which the norm then sees 12 at most.
template <int DT>
__device__ __forceinline__ float chunk_sumsq(const ClipChunk& T, int tid) {
  const int n = T.n;
  constexpr int K = Vec16<DT>::kElems;
  float2 s[2] = {};
  int done = 0;
  const void* base = T.grad;
  if (T.vec) {
    const uint4* p = static_cast<const uint4*>(base);
    const int nv = n / K;
#pragma unroll 4
    for (int i = tid; i < nv; i += kThreads) {
      float2 f[K / 2];
      Vec16<DT>::unpack(p[i], f);
#pragma unroll
      for (int j = 0; j < K / 2; ++j) s[j & 1] = fma2(f[j], f[j], s[j & 1]);
    }
    done = nv * K;
  }
  int i = done + tid;
  for (; i + 3 * kThreads < n; i += 4 * kThreads) {
    float2 f[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      f[j] = make_float2(load_elem<DT>(base, i + 2 * j * kThreads), load_elem<DT>(base, i + (2 * j + 1) * kThreads));
#pragma unroll
    for (int j = 0; j < 2; ++j) s[j] = fma2(f[j], f[j], s[j]);
  }
  for (; i < n; i += kThreads) {
    const float f = load_elem<DT>(base, i);
    s[0].x = fmaf(f, f, s[0].x);
  }
  return (s[0].x + s[0].y) + (s[1].x + s[1].y);
}

// One read: 872M bf16 elements in 258 us, 6.76 TB/s.  A few elements are bound
// by latency: 24 vectors of 4096 take 5 us, most of it the two reductions.
__global__ void __launch_bounds__(kThreads) clip_norm_kernel(const ClipLaunch L) {
  __shared__ double s_warp[kThreads / 32];
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  double acc = 0.0;
  depends_wait();
  for (int c = blockIdx.x; c < L.n_chunks; c += gridDim.x) {
    const ClipChunk T = L.chunks[c];
    const float s = T.dtype == QMUON_BF16   ? chunk_sumsq<QMUON_BF16>(T, tid)
                    : T.dtype == QMUON_FP16 ? chunk_sumsq<QMUON_FP16>(T, tid)
                                            : chunk_sumsq<QMUON_FP32>(T, tid);
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
__device__ __forceinline__ void chunk_scale(const ClipChunk& T, int tid, float c) {
  const int n = T.n;
  constexpr int K = Vec16<DT>::kElems;
  int done = 0;
  void* base = T.grad;
  if (T.vec) {
    uint4* p = static_cast<uint4*>(base);
    const int nv = n / K;
#pragma unroll 4
    for (int i = tid; i < nv; i += kThreads) {
      float2 f[K / 2];
      Vec16<DT>::unpack(p[i], f);
#pragma unroll
      for (int j = 0; j < K / 2; ++j) f[j] = mul2_rn(f[j], c);
      p[i] = Vec16<DT>::pack(f);
    }
    done = nv * K;
  }
  for (int i = done + tid; i < n; i += kThreads) store_elem<DT>(base, i, load_elem<DT>(base, i) * c);
}

// Another read and a write, at 7.1 TB/s.
__global__ void __launch_bounds__(kThreads) clip_scale_kernel(const ClipLaunch L) {
  // the last chunks first: L2 still holds them from the norm
  const ClipChunk T = L.chunks[gridDim.x - 1 - blockIdx.x];
  depends_wait();
  const float c = __ldcg(L.norm + 1);
  if (!(c < 1.0f)) return;   // within the bound, or not finite
  if (T.dtype == QMUON_BF16) chunk_scale<QMUON_BF16>(T, threadIdx.x, c);
  else if (T.dtype == QMUON_FP16) chunk_scale<QMUON_FP16>(T, threadIdx.x, c);
  else chunk_scale<QMUON_FP32>(T, threadIdx.x, c);
}

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------
// With g' = c g (c the clipping coefficient), every operation rounded once:
//   m <- b1 m + (1 - b1) g'          v <- b2 v + (1 - b2) g'^2
//   p <- p (1 - lr wd) - (lr / (1 - b1^t)) (m / (sqrt(v) / sqrt(1 - b2^t) + eps))
constexpr int kWarps = kThreads / 32;
constexpr int kAdamChunk = 2048;   // elements with fp32 states: 8 per thread
// With 8-bit states a chunk is J blocks of 256 per warp: 3, or 1 where 3 would
// leave SMs without a CTA (fewer than two chunks per SM).
constexpr int kManyBlocks = 3;

struct AdamTensor {
  float* param;
  const void* grad;
  void* copy;          // 16-bit copy of the parameters, or null
  void* m;
  void* v;
  float* m_absmax;     // 8-bit states
  float* v_absmax;
  int64_t end;         // elements are [begin, end) of the arrays, which point `begin` elements
  int32_t begin;       //   before the caller's: 0..3, so that quads of elements are aligned
  int32_t first_chunk;
  float lr_scale, weight_decay;
  int32_t index;       // in the caller's list: the stochastic rounding's counter
  int16_t grad_dtype, copy_dtype;
  int32_t vec;         // quads are aligned in every array
};

struct AdamLaunch {
  const AdamTensor* tensors;
  const int32_t* chunk_tensor;
  const float* grad_scale;   // D, or null
  float lr, b1, omb1, b2, omb2, rbc1, rbc2, eps;
  uint32_t step;
  PhiloxKeys keys;
};

struct AdamCoef {
  float scale, decay, step;
};

__device__ __forceinline__ AdamCoef adam_coef(const AdamLaunch& L, const AdamTensor& T, float scale) {
  const float lr = __fmul_rn(L.lr, T.lr_scale);
  return {scale, __fsub_rn(1.0f, __fmul_rn(lr, T.weight_decay)), __fmul_rn(lr, L.rbc1)};
}

// 1 / x to 1 ulp for normal x below 2^126 (zero above).
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two elements: the new momentum, parameter and square root of the new second
// moment, from the old momentum, parameter and second moment.  Only the
// quotient is not correctly rounded (2 ulp): it reaches the parameter alone,
// scaled by the step size.
__device__ __forceinline__ void adam_pair(const AdamLaunch& L, const AdamCoef& C, float2 g, float2& p, float2& m, float2& v,
                                          float2& r) {
  g = mul2_rn(g, C.scale);
  const float2 mb = mul2_rn(m, L.b1), mg = mul2_rn(g, L.omb1);
  const float2 vb = mul2_rn(v, L.b2), vg = mul2_rn(mul2_rn(g, g), L.omb2);
  m = make_float2(__fadd_rn(mb.x, mg.x), __fadd_rn(mb.y, mg.y));
  v = make_float2(__fadd_rn(vb.x, vg.x), __fadd_rn(vb.y, vg.y));
  r = make_float2(__fsqrt_rn(v.x), __fsqrt_rn(v.y));
  const float2 d = mul2_rn(r, L.rbc2);
  const float2 u = mul2_rn(mul2_rn(m, make_float2(rcp_approx(__fadd_rn(d.x, L.eps)), rcp_approx(__fadd_rn(d.y, L.eps)))), C.step);
  const float2 q = mul2_rn(p, C.decay);
  p = make_float2(__fsub_rn(q.x, u.x), __fsub_rn(q.y, u.y));
}

// One CTA per chunk, two quads of elements per thread.  A CTA that takes its
// chunk and leaves keeps DRAM busier than one that stays: the same traffic
// without any arithmetic runs at 7.06 TB/s with one CTA per 2048 elements and at
// 6.4 with the resident CTAs looping over chunks (2^28 elements), rings of
// asynchronous copies ahead of them or not.  What is left is DRAM: 419M elements
// with fp32 states, bf16 gradients and a bf16 copy take 1656 us (7.09 TB/s), with
// 8-bit states 995 us (6.77 TB/s).  Chunks that lie wholly inside a
// tensor whose arrays are aligned (AdamTensor::vec) move in vectors; in the
// chunks at a tensor's ends, and in all of an unaligned one, quads that are not
// whole move element by element.
struct Quad {
  float2 a, b;
};

__device__ __forceinline__ Quad as_quad(const float4& t) { return {make_float2(t.x, t.y), make_float2(t.z, t.w)}; }
__device__ __forceinline__ Quad load_quad(const float* p) { return as_quad(__ldcs(reinterpret_cast<const float4*>(p))); }
template <int GDT>
__device__ __forceinline__ Quad load_grad(const void* g, int64_t e) {
  if constexpr (GDT == QMUON_FP32) return load_quad(static_cast<const float*>(g) + e);
  else {
    const uint2 w = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(g) + e));
    return {unpack2<GDT>(w.x), unpack2<GDT>(w.y)};
  }
}
__device__ __forceinline__ Quad load_grad(const AdamTensor& T, int64_t e) {
  return T.grad_dtype == QMUON_FP32   ? load_grad<QMUON_FP32>(T.grad, e)
         : T.grad_dtype == QMUON_BF16 ? load_grad<QMUON_BF16>(T.grad, e)
                                      : load_grad<QMUON_FP16>(T.grad, e);
}
__device__ __forceinline__ float grad_elem(const AdamTensor& T, int64_t e) {
  if (T.grad_dtype == QMUON_FP32) return load_elem<QMUON_FP32>(T.grad, e);
  if (T.grad_dtype == QMUON_BF16) return load_elem<QMUON_BF16>(T.grad, e);
  return load_elem<QMUON_FP16>(T.grad, e);
}
constexpr int kNoCopy = -1;
template <int CDT>
__device__ __forceinline__ void store_copy_quad(uint16_t* c, const Quad& p) {
  if constexpr (CDT != kNoCopy)
    __stcs(reinterpret_cast<uint2*>(c), make_uint2(pack2<CDT>(p.a.x, p.a.y), pack2<CDT>(p.b.x, p.b.y)));
}
__device__ __forceinline__ void store_quad(float* d, const Quad& q) {
  __stcs(reinterpret_cast<float4*>(d), make_float4(q.a.x, q.a.y, q.b.x, q.b.y));
}
__device__ __forceinline__ void store_param_quad(const AdamTensor& T, int64_t e, const Quad& p) {
  store_quad(T.param + e, p);
  uint16_t* c = static_cast<uint16_t*>(T.copy) + e;
  if (!T.copy) return;
  if (T.copy_dtype == QMUON_BF16) store_copy_quad<QMUON_BF16>(c, p);
  else store_copy_quad<QMUON_FP16>(c, p);
}
__device__ __forceinline__ void store_param_elem(const AdamTensor& T, int64_t e, float p) {
  T.param[e] = p;
  if (!T.copy) return;
  if (T.copy_dtype == QMUON_BF16) store_elem<QMUON_BF16>(T.copy, e, p);
  else store_elem<QMUON_FP16>(T.copy, e, p);
}

// One element with fp32 states, from and to memory.
__device__ __forceinline__ void adam_single(const AdamLaunch& L, const AdamTensor& T, const AdamCoef& C, int64_t e) {
  float* mp = static_cast<float*>(T.m) + e;
  float* vp = static_cast<float*>(T.v) + e;
  float2 p = make_float2(T.param[e], 0.0f), m = make_float2(*mp, 0.0f), v = make_float2(*vp, 0.0f), r;
  adam_pair(L, C, make_float2(grad_elem(T, e), 0.0f), p, m, v, r);
  store_param_elem(T, e, p.x);
  *mp = m.x;
  *vp = v.x;
}

// Calls f with the gradient's and the copy's type as constants.
template <class F>
__device__ __forceinline__ void with_types(const AdamTensor& T, F&& f) {
  auto copy = [&](auto g) {
    if (!T.copy) f(g, std::integral_constant<int, kNoCopy>{});
    else if (T.copy_dtype == QMUON_BF16) f(g, std::integral_constant<int, QMUON_BF16>{});
    else f(g, std::integral_constant<int, QMUON_FP16>{});
  };
  if (T.grad_dtype == QMUON_FP32) copy(std::integral_constant<int, QMUON_FP32>{});
  else if (T.grad_dtype == QMUON_BF16) copy(std::integral_constant<int, QMUON_BF16>{});
  else copy(std::integral_constant<int, QMUON_FP16>{});
}

// Calls f(T, C, c) for this CTA's chunk: chunk c of tensor T, by reference into
// the plan's table.
template <class F>
__device__ __forceinline__ void for_chunk(const AdamLaunch& L, F&& f) {
  const AdamTensor& T = L.tensors[__ldg(L.chunk_tensor + blockIdx.x)];
  depends_wait();
  const float scale = L.grad_scale ? __ldcg(L.grad_scale) : 1.0f;
  if (isfinite(scale)) f(T, scale, (int)blockIdx.x - T.first_chunk);
}

// ---- fp32 states ----
template <int GDT, int CDT>
__device__ __forceinline__ void f32_fast(const AdamLaunch& L, const AdamTensor& T, const AdamCoef& C, int c) {
  constexpr int kHalf = kThreads * 4;
  const int64_t e = (int64_t)c * kAdamChunk + threadIdx.x * 4;   // of the first quad; the second is kHalf on
  float* p = T.param + e;
  float* m = static_cast<float*>(T.m) + e;
  float* v = static_cast<float*>(T.v) + e;
  Quad P[2], M[2], V[2], G[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    G[k] = load_grad<GDT>(T.grad, e + k * kHalf);
    P[k] = load_quad(p + k * kHalf);
    M[k] = load_quad(m + k * kHalf);
    V[k] = load_quad(v + k * kHalf);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float2 r;
    adam_pair(L, C, G[k].a, P[k].a, M[k].a, V[k].a, r);
    adam_pair(L, C, G[k].b, P[k].b, M[k].b, V[k].b, r);
    store_quad(p + k * kHalf, P[k]);
    store_quad(m + k * kHalf, M[k]);
    store_quad(v + k * kHalf, V[k]);
    store_copy_quad<CDT>(static_cast<uint16_t*>(T.copy) + e + k * kHalf, P[k]);
  }
}

__device__ __noinline__ void f32_slow(const AdamLaunch& L, const AdamTensor& in_table, float scale, int c) {
  const AdamTensor T = in_table;
  const AdamCoef C = adam_coef(L, T, scale);
  const int t = threadIdx.x;
  const int64_t e0 = (int64_t)c * kAdamChunk;
  if (!T.vec) {   // neighbouring threads on neighbouring elements
#pragma unroll 4
    for (int j = 0; j < kAdamChunk / kThreads; ++j) {
      const int64_t e = e0 + j * kThreads + t;
      if (e < T.end) adam_single(L, T, C, e);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t e = e0 + (k * kThreads + t) * 4;
    if (e >= T.begin && e + 4 <= T.end) {
      float4* mp = reinterpret_cast<float4*>(static_cast<float*>(T.m) + e);
      float4* vp = reinterpret_cast<float4*>(static_cast<float*>(T.v) + e);
      Quad P = load_quad(T.param + e), M = as_quad(__ldcs(mp)), V = as_quad(__ldcs(vp));
      const Quad G = load_grad(T, e);
      float2 r;
      adam_pair(L, C, G.a, P.a, M.a, V.a, r);
      adam_pair(L, C, G.b, P.b, M.b, V.b, r);
      store_param_quad(T, e, P);
      store_quad(reinterpret_cast<float*>(mp), M);
      store_quad(reinterpret_cast<float*>(vp), V);
    } else {
      for (int j = 0; j < 4; ++j)
        if (e + j >= T.begin && e + j < T.end) adam_single(L, T, C, e + j);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 4) adamw_f32_kernel(const __grid_constant__ AdamLaunch L) {
  for_chunk(L, [&](const AdamTensor& in_table, float scale, int c) {
    const AdamTensor T = in_table;
    const AdamCoef C = adam_coef(L, T, scale);
    if (T.vec && (c > 0 || T.begin == 0) && (int64_t)(c + 1) * kAdamChunk <= T.end)
      with_types(T, [&](auto g, auto k) { f32_fast<decltype(g)::value, decltype(k)::value>(L, T, C, c); });
    else
      f32_slow(L, in_table, scale, c);
  });
}

// ---- 8-bit states ----
// m and r = sqrt(v) are E4M3 codes with one fp32 maximum per 256 elements:
// x = code * (max / 448).  The root is stored, not v: its codes then cover as
// many powers of two as the momentum's.  A root above zero takes at least code
// 1: the two maxima decay at different rates and m and r round on their own, so
// that r may round to zero where m does not, and the next step would divide that
// m by eps alone (a block with one gradient of 10 and, 49 steps later, another
// element's of 1e-5 then moved that one by 90 lr).
//
// A warp takes a block, lane l its elements 4l..4l+3 and 128+4l..128+4l+3: every
// load and store of the warp is one contiguous run, and a quad of elements
// shares a random counter.

// E4M3 of four scaled values with 16 random bits each: rounded up in magnitude
// with probability (remainder / step) to 2^-16.  2^-120 |x| has its exponent
// field where the code's is, subnormals included, so the bits above the lowest
// 20 are the code; it is cut, not rounded, to the 20 that a subnormal code's
// remainder keeps, as a remainder that misses a whole step with its random bits
// must not be rounded up to one.  The largest value's code, 0x7E with all lower bits zero (up
// to an ulp), cannot be carried to 0x7F by random bits of which the lowest four
// are zero: 0x7F remains for NaN alone.
template <bool SIGNED>
__device__ __forceinline__ uint32_t encode_sr4(const Quad& x, uint32_t u0, uint32_t u1, uint32_t u2, uint32_t u3) {
  constexpr float kShift = 7.52316384526264e-37f;   // 2^-120
  const float2 a = mul2_rz(x.a, kShift), b = mul2_rz(x.b, kShift);
  auto code = [](float y, uint32_t u) { return min(__float_as_uint(fabsf(y)) + u, 0x7F00000u) << 4; };
  const uint32_t c0 = code(a.x, u0), c1 = code(a.y, u1), c2 = code(b.x, u2), c3 = code(b.y, u3);
  const uint32_t w = __byte_perm(__byte_perm(c0, c1, 0x0073u), __byte_perm(c2, c3, 0x0073u), 0x5410u);
  if constexpr (!SIGNED) return w;
  const uint32_t s = __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0073u),
                                 __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0073u), 0x5410u);
  return w | (s & 0x80808080u);
}

// Code 1 for those of a quad's scaled roots that are above zero and have code 0,
// to nearest: few words hold a zero byte, so the test for one (exact in whether
// there is any) is all that most quads pay, and no time (419M elements 988 us with
// and without).  Stochastically the roots are raised to code 1's value first: the
// test, which keeps them in registers until after the random numbers, takes 97 us
// for 35M elements, this 95.5, neither 94.6.
__device__ __forceinline__ uint32_t root_codes(uint32_t w, const Quad& r) {
  if ((w - 0x01010101u) & ~w & 0x80808080u) {
    if ((w & 0xFFu) == 0 && r.a.x > 0.0f) w |= 0x1u;
    if ((w & 0xFF00u) == 0 && r.a.y > 0.0f) w |= 0x100u;
    if ((w & 0xFF0000u) == 0 && r.b.x > 0.0f) w |= 0x10000u;
    if ((w & 0xFF000000u) == 0 && r.b.y > 0.0f) w |= 0x1000000u;
  }
  return w;
}

__device__ __forceinline__ float2 at_least_code1(float2 x) {   // a NaN stays
  constexpr float k1 = 0.001953125f;   // 2^-9
  return make_float2(x.x > 0.0f ? fmaxf(x.x, k1) : x.x, x.y > 0.0f ? fmaxf(x.y, k1) : x.y);
}

// Two quads of a block in a lane.
struct E4m3Quads {
  Quad p[2], g[2], m[2], r[2];
  uint32_t mc[2], vc[2];
  float m_max, r_max;
};

// Decodes a block, updates it and encodes it under its new maxima, in which
// only the n[k] elements of each quad that exist take part.
template <bool SR, bool WHOLE>
__device__ __forceinline__ void e4m3_update(const AdamLaunch& L, const AdamCoef& C, E4m3Quads& q, const int* n, int64_t e0,
                                            int32_t index) {
  const float m_unit = __fdiv_rn(q.m_max, 448.0f), r_unit = __fdiv_rn(q.r_max, 448.0f);
  float m_max = 0.0f, r_max = 0.0f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    Quad &m = q.m[k], &r = q.r[k];
    m.a = mul2_rn(e4m3x2_to(q.mc[k]), m_unit);
    m.b = mul2_rn(e4m3x2_to(q.mc[k] >> 16), m_unit);
    const float2 ra = mul2_rn(e4m3x2_to(q.vc[k]), r_unit), rb = mul2_rn(e4m3x2_to(q.vc[k] >> 16), r_unit);
    float2 va = mul2_rn(ra, ra), vb = mul2_rn(rb, rb);
    adam_pair(L, C, q.g[k].a, q.p[k].a, m.a, va, r.a);
    adam_pair(L, C, q.g[k].b, q.p[k].b, m.b, vb, r.b);
    if constexpr (!WHOLE) {
      if (n[k] < 1) m.a.x = r.a.x = 0.0f;
      if (n[k] < 2) m.a.y = r.a.y = 0.0f;
      if (n[k] < 3) m.b.x = r.b.x = 0.0f;
      if (n[k] < 4) m.b.y = r.b.y = 0.0f;
    }
    m_max = fmaxf(m_max, fmaxf(fmaxf(fabsf(m.a.x), fabsf(m.a.y)), fmaxf(fabsf(m.b.x), fabsf(m.b.y))));
    r_max = fmaxf(r_max, fmaxf(fmaxf(r.a.x, r.a.y), fmaxf(r.b.x, r.b.y)));
  }
  q.m_max = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m_max)));   // not negative: ordered as integers
  q.r_max = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(r_max)));
  constexpr float kMax = 3.402823466e+38f;   // a zero or tiny maximum: no infinite factor
  const float m_sc = fminf(__fdiv_rn(448.0f, q.m_max), kMax), r_sc = fminf(__fdiv_rn(448.0f, q.r_max), kMax);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float2 ma = mul2_rn(q.m[k].a, m_sc), mb = mul2_rn(q.m[k].b, m_sc), ra = mul2_rn(q.r[k].a, r_sc), rb = mul2_rn(q.r[k].b, r_sc);
    if constexpr (SR) {
      const uint64_t j = (uint64_t)(e0 + 128 * k) >> 2;
      const uint4 w = philox(make_uint4((uint32_t)j, (uint32_t)(j >> 32), (uint32_t)index, L.step), L.keys);
      // per element: the word's low half for m, its high half for r, above four zero bits
      auto lo = [](uint32_t x) { return (x << 4) & 0xFFFF0u; };
      auto hi = [](uint32_t x) { return (x >> 12) & 0xFFFF0u; };
      q.mc[k] = encode_sr4<true>({ma, mb}, lo(w.x), lo(w.y), lo(w.z), lo(w.w));
      q.vc[k] = encode_sr4<false>({at_least_code1(ra), at_least_code1(rb)}, hi(w.x), hi(w.y), hi(w.z), hi(w.w));
    } else {
      q.mc[k] = cvt_e4m3x2(ma.x, ma.y) | (cvt_e4m3x2(mb.x, mb.y) << 16);
      q.vc[k] = root_codes(cvt_e4m3x2(ra.x, ra.y) | (cvt_e4m3x2(rb.x, rb.y) << 16), {ra, rb});
    }
  }
}

// One block's inputs in shared memory, as its warp's asynchronous copies
// bring them: all in 16-byte pieces but the two maxima.
template <int GDT>
struct __align__(16) E4m3Stage {
  float p[kBlock];
  unsigned char g[kBlock * elem_size(GDT)];
  uint8_t codes[2][kBlock];   // m, v
  float maxima[4];
};

// J whole blocks per warp, all of their loads in flight from the start: the
// copies need no registers while they are.  With one block per warp, loaded
// into registers, the arithmetic (54 instructions per element, 77 with random
// numbers) left too few bytes in flight.  2^28 elements with a copy took 776 us
// so, 680 with J = 2, 653 with 3, 647 with 4; rounded stochastically 743, 688 and
// 713, where the arithmetic is the bound.  With the tensor's record in registers
// 638 (6.75 TB/s) and 667.
template <int GDT, int CDT, bool SR, int J>
__device__ __forceinline__ void e4m3_fast(const AdamLaunch& L, const AdamTensor& T, const AdamCoef& C, int64_t first, int n,
                                          unsigned char* smem) {
  static_assert(J <= 3, "one wait per block in flight below");
  constexpr int kGs = elem_size(GDT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  E4m3Stage<GDT>* ring = reinterpret_cast<E4m3Stage<GDT>*>(smem) + warp;
  n = (n - warp + kWarps - 1) / kWarps;   // this warp's: blocks first + warp, first + warp + 8, ..
  int64_t blk = first + warp;
  const unsigned char* code_src = static_cast<const unsigned char*>(lane < 16 ? T.m : T.v) + (lane & 15) * 16;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (j < n) {
      E4m3Stage<GDT>& S = ring[j * kWarps];
      const int64_t e = (blk + j * kWarps) * kBlock;
#pragma unroll
      for (int k = 0; k < 2; ++k) async16(&S.p[(k * 32 + lane) * 4], T.param + e + (k * 32 + lane) * 4);
#pragma unroll
      for (int k = 0; k < kGs / 2; ++k)
        async16(&S.g[(k * 32 + lane) * 16], static_cast<const unsigned char*>(T.grad) + e * kGs + (k * 32 + lane) * 16);
      async16(&S.codes[0][lane * 16], code_src + e);
      if (lane < 2) async4(&S.maxima[lane], (lane == 0 ? T.m_absmax : T.v_absmax) + blk + j * kWarps);
    }
    async_commit();
  }
#pragma unroll 1
  for (int j = 0; j < n; ++j, blk += kWarps) {
    if (j == J - 1) async_wait<0>();
    else if (j == J - 2) async_wait<1>();
    else async_wait<2>();
    __syncwarp();   // the other lanes' copies
    const E4m3Stage<GDT>& S = ring[j * kWarps];
    const int64_t e = blk * kBlock + 4 * lane;   // of the first quad; the second is 128 on
    E4m3Quads q;
    q.m_max = S.maxima[0];
    q.r_max = S.maxima[1];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = 128 * k + 4 * lane;
      q.p[k] = as_quad(*reinterpret_cast<const float4*>(&S.p[i]));
      if constexpr (kGs == 4) {
        q.g[k] = as_quad(*reinterpret_cast<const float4*>(&S.g[i * 4]));
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(&S.g[i * 2]);
        q.g[k] = {unpack2<GDT>(w.x), unpack2<GDT>(w.y)};
      }
      q.mc[k] = *reinterpret_cast<const uint32_t*>(&S.codes[0][i]);
      q.vc[k] = *reinterpret_cast<const uint32_t*>(&S.codes[1][i]);
    }
    e4m3_update<SR, true>(L, C, q, nullptr, e, T.index);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(T.m) + e + 128 * k), q.mc[k]);
      __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(T.v) + e + 128 * k), q.vc[k]);
      store_quad(T.param + e + 128 * k, q.p[k]);
      store_copy_quad<CDT>(static_cast<uint16_t*>(T.copy) + e + 128 * k, q.p[k]);
    }
    if (lane < 2) (lane == 0 ? T.m_absmax : T.v_absmax)[blk] = lane == 0 ? q.m_max : q.r_max;
  }
}

// One block, whole or not, by the calling warp.
template <bool SR>
__device__ __noinline__ void e4m3_slow(const AdamLaunch& L, const AdamTensor& in_table, float scale, int64_t blk) {
  const AdamTensor T = in_table;
  const AdamCoef C = adam_coef(L, T, scale);
  const int lane = threadIdx.x & 31;
  const int64_t e0 = blk * kBlock + 4 * lane;
  uint8_t* mp = static_cast<uint8_t*>(T.m) + e0;
  uint8_t* vp = static_cast<uint8_t*>(T.v) + e0;
  E4m3Quads q;
  int n[2];
  q.m_max = T.m_absmax[blk];
  q.r_max = T.v_absmax[blk];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t e = e0 + 128 * k;
    n[k] = (int)max((int64_t)0, min((int64_t)4, T.end - e));
    if (T.vec && n[k] == 4) {
      q.p[k] = load_quad(T.param + e);
      q.g[k] = load_grad(T, e);
      q.mc[k] = *reinterpret_cast<const uint32_t*>(mp + 128 * k);
      q.vc[k] = *reinterpret_cast<const uint32_t*>(vp + 128 * k);
    } else {
      float pe[4], ge[4];
      q.mc[k] = q.vc[k] = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        pe[j] = ge[j] = 0.0f;
        if (j >= n[k]) continue;
        pe[j] = T.param[e + j];
        ge[j] = grad_elem(T, e + j);
        q.mc[k] |= (uint32_t)mp[128 * k + j] << (8 * j);
        q.vc[k] |= (uint32_t)vp[128 * k + j] << (8 * j);
      }
      q.p[k] = {make_float2(pe[0], pe[1]), make_float2(pe[2], pe[3])};
      q.g[k] = {make_float2(ge[0], ge[1]), make_float2(ge[2], ge[3])};
    }
  }
  e4m3_update<SR, false>(L, C, q, n, e0, T.index);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (T.vec && n[k] == 4) {
      *reinterpret_cast<uint32_t*>(mp + 128 * k) = q.mc[k];
      *reinterpret_cast<uint32_t*>(vp + 128 * k) = q.vc[k];
      store_param_quad(T, e0 + 128 * k, q.p[k]);
    } else {
      const float pe[4] = {q.p[k].a.x, q.p[k].a.y, q.p[k].b.x, q.p[k].b.y};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= n[k]) continue;
        mp[128 * k + j] = (uint8_t)(q.mc[k] >> (8 * j));
        vp[128 * k + j] = (uint8_t)(q.vc[k] >> (8 * j));
        store_param_elem(T, e0 + 128 * k + j, pe[j]);
      }
    }
  }
  if (lane == 0) {
    T.m_absmax[blk] = q.m_max;
    T.v_absmax[blk] = q.r_max;
  }
}

template <bool SR, int J>
__global__ void __launch_bounds__(kThreads, 4) adamw_e4m3_kernel(const __grid_constant__ AdamLaunch L) {
  extern __shared__ __align__(16) unsigned char smem[];
  for_chunk(L, [&](const AdamTensor& in_table, float scale, int c) {
    const AdamTensor T = in_table;
    const AdamCoef C = adam_coef(L, T, scale);
    constexpr int kPer = J * kWarps;
    const int64_t first = (int64_t)c * kPer, nb = (T.end + kBlock - 1) / kBlock;
    const int whole = T.vec ? (int)min((int64_t)kPer, T.end / kBlock - first) : 0, all = (int)min((int64_t)kPer, nb - first);
    if (whole > 0)
      with_types(T, [&](auto g, auto k) { e4m3_fast<decltype(g)::value, decltype(k)::value, SR, J>(L, T, C, first, whole, smem); });
    for (int b = whole + (int)(threadIdx.x >> 5); b < all; b += kWarps) e4m3_slow<SR>(L, in_table, scale, first + b);
  });
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool is_dtype(int v) { return v == QMUON_BF16 || v == QMUON_FP16 || v == QMUON_FP32; }

using AdamKernel = void (*)(AdamLaunch);
AdamKernel adam_kernel(qmuon_state_kind state, bool sr, int per_warp) {
  if (state == QMUON_STATE_F32) return adamw_f32_kernel;
  if (per_warp == 1) return sr ? adamw_e4m3_kernel<true, 1> : adamw_e4m3_kernel<false, 1>;
  return sr ? adamw_e4m3_kernel<true, kManyBlocks> : adamw_e4m3_kernel<false, kManyBlocks>;
}
// The chunks' table: for each chunk of `chunk` elements, the position of its
// tensor among the non-empty ones.
struct Chunks {
  std::vector<int32_t> tensor;
  std::vector<int32_t> first;   // per non-empty tensor
  bool add(int64_t numel, int64_t chunk) {
    const int64_t k = (numel + chunk - 1) / chunk;
    if ((int64_t)tensor.size() + k > kMaxChunks) return false;
    first.push_back((int32_t)tensor.size());
    tensor.insert(tensor.end(), (size_t)k, (int32_t)first.size() - 1);
    return true;
  }
};

// One device allocation holding [256 zero bytes | tensors | chunk table].
template <class Tensor>
cudaError_t upload(const std::vector<Tensor>& ts, const std::vector<int32_t>& chunks, void** table, Tensor** d_ts,
                   int32_t** d_chunks) {
  constexpr size_t head = 256;
  const size_t tb = (ts.size() * sizeof(Tensor) + 255) / 256 * 256;
  std::vector<unsigned char> blob(head + tb + chunks.size() * 4, 0);
  std::memcpy(blob.data() + head, ts.data(), ts.size() * sizeof(Tensor));
  if (!chunks.empty()) std::memcpy(blob.data() + head + tb, chunks.data(), chunks.size() * 4);
  cudaError_t e = cudaMalloc(table, blob.size());
  if (e != cudaSuccess) return e;
  e = upload_and_wait(*table, blob.data(), blob.size());
  if (e != cudaSuccess) {
    cudaFree(*table);
    *table = nullptr;
    return e;
  }
  unsigned char* b = static_cast<unsigned char*>(*table);
  *d_ts = reinterpret_cast<Tensor*>(b + head);
  if (d_chunks) *d_chunks = reinterpret_cast<int32_t*>(b + head + tb);
  return cudaSuccess;
}

}  // namespace
}  // namespace qm

using namespace qm;

struct qmuon_clip_plan {
  void* table = nullptr;   // the ticket is its first word
  ClipChunk* chunks = nullptr;
  int32_t n_chunks = 0;
  int32_t grid = 0;
};

struct qmuon_adamw_plan {
  void* table = nullptr;
  AdamTensor* tensors = nullptr;
  int32_t* chunk_tensor = nullptr;
  int32_t n_chunks = 0;
  int32_t per_warp = 0;    // J
  int32_t smem = 0;
  qmuon_state_kind state = QMUON_STATE_F32;
};

extern "C" qmuon_status qmuon_clip_plan_create(const qmuon_grad* grads, int32_t n, qmuon_clip_plan** out) {
  NvtxRange nvtx_range("qmuon_clip_plan_create");
  return no_throw("qmuon_clip_plan_create", [&]() -> qmuon_status {
    if (!out) return QMUON_ERR_INVALID_ARGUMENT;
    *out = nullptr;
    if (!grads || n <= 0) return QMUON_ERR_INVALID_ARGUMENT;
    std::vector<ClipChunk> chunks;
    for (int32_t i = 0; i < n; ++i) {
      const qmuon_grad& g = grads[i];
      if (!is_dtype(g.dtype) || g.numel < 0 || g.numel > kMaxElems) return QMUON_ERR_INVALID_ARGUMENT;
      if (g.numel == 0) continue;
      if (!g.grad || !is_aligned(g.grad, elem_size(g.dtype))) return QMUON_ERR_INVALID_ARGUMENT;
      if ((int64_t)chunks.size() + (g.numel + kClipChunk - 1) / kClipChunk > kMaxChunks) return QMUON_ERR_INVALID_ARGUMENT;
      for (int64_t e = 0; e < g.numel; e += kClipChunk)
        chunks.push_back({static_cast<unsigned char*>(g.grad) + e * elem_size(g.dtype),
                          (int32_t)std::min<int64_t>(g.numel - e, kClipChunk), (int16_t)g.dtype,
                          (int16_t)is_aligned(g.grad, 16)});
    }
    if (chunks.empty()) return QMUON_ERR_INVALID_ARGUMENT;
    std::unique_ptr<qmuon_clip_plan> P(new qmuon_clip_plan);
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, clip_norm_kernel, kThreads, 0);
    if (e != cudaSuccess) return set_error("qmuon_clip_plan_create (device)", e);
    P->n_chunks = (int32_t)chunks.size();
    P->grid = std::min(P->n_chunks, sms * std::max(per_sm, 1));
    e = upload(chunks, {}, &P->table, &P->chunks, nullptr);
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
  L.chunks = plan->chunks;
  L.n_chunks = plan->n_chunks;
  L.ticket = static_cast<unsigned int*>(plan->table);
  L.partials = static_cast<double*>(ws);
  L.norm = norm;
  L.max_norm = max_norm;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_dependent(clip_norm_kernel, plan->grid, kThreads, 0, s, L);
  if (e == cudaSuccess && apply) e = launch_dependent(clip_scale_kernel, plan->n_chunks, kThreads, 0, s, L);
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
    bool f32_grads = false;
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
      // fp32 states: arrays that are slices of flat buffers at one element offset become aligned together after a
      // head of up to three elements (8-bit blocks count from the first element and start on 16 bytes)
      int begin = 0;
      bool vec = false;
      for (; !vec && begin < (f32 ? 4 : 1); ++begin) {
        auto at = [&](const void* p, size_t es) { return reinterpret_cast<uintptr_t>(p) - begin * es; };
        vec = at(t.param, 4) % 16 == 0 && at(t.grad, gs) % (f32 ? 4 * gs : 16) == 0 && (!t.copy || at(t.copy, 2) % 8 == 0) &&
              (!f32 || (at(t.m, 4) % 16 == 0 && at(t.v, 4) % 16 == 0));
      }
      begin = vec ? begin - 1 : 0;
      auto back = [&](auto* p, size_t es) {
        return p ? reinterpret_cast<decltype(p)>(reinterpret_cast<uintptr_t>(p) - begin * es) : nullptr;
      };
      AdamTensor a{};
      a.param = back(t.param, 4);
      a.grad = back(t.grad, gs);
      a.copy = back(t.copy, 2);
      a.m = back(t.m, 4);
      a.v = back(t.v, 4);
      a.m_absmax = t.m_absmax;
      a.v_absmax = t.v_absmax;
      a.begin = begin;
      a.end = t.numel + begin;
      a.lr_scale = t.lr_scale;
      a.weight_decay = t.weight_decay;
      a.index = i;
      a.grad_dtype = (int16_t)t.grad_dtype;
      a.copy_dtype = (int16_t)t.copy_dtype;
      a.vec = vec;
      f32_grads = f32_grads || t.grad_dtype == QMUON_FP32;
      ts.push_back(a);
    }
    if (ts.empty()) return QMUON_ERR_INVALID_ARGUMENT;
    std::unique_ptr<qmuon_adamw_plan> P(new qmuon_adamw_plan);
    P->state = state;
    int64_t chunk = kAdamChunk;
    cudaError_t e = cudaSuccess;
    if (!f32) {
      int dev = 0, sms = 0;
      e = cudaGetDevice(&dev);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
      int64_t many = 0;
      for (const AdamTensor& a : ts) many += (a.end + kManyBlocks * kWarps * kBlock - 1) / (kManyBlocks * kWarps * kBlock);
      P->per_warp = many >= 2 * (int64_t)sms ? kManyBlocks : 1;
      chunk = (int64_t)P->per_warp * kWarps * kBlock;
      P->smem = P->per_warp * kWarps * (int)(f32_grads ? sizeof(E4m3Stage<QMUON_FP32>) : sizeof(E4m3Stage<QMUON_BF16>));
      for (int sr = 0; sr < 2 && e == cudaSuccess; ++sr)
        e = cudaFuncSetAttribute(adam_kernel(state, sr != 0, P->per_warp), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kManyBlocks * kWarps * (int)sizeof(E4m3Stage<QMUON_FP32>));
      if (e != cudaSuccess) return set_error("qmuon_adamw_plan_create (device)", e);
    }
    Chunks ch;
    for (AdamTensor& a : ts) {
      if (!ch.add(a.end, chunk)) return QMUON_ERR_INVALID_ARGUMENT;
      a.first_chunk = ch.first.back();
    }
    P->n_chunks = (int32_t)ch.tensor.size();
    e = upload(ts, ch.tensor, &P->table, &P->tensors, &P->chunk_tensor);
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
  // as the kernels take them, in fp32
  if (!(std::fabs(lr) <= FLT_MAX) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0))
    return QMUON_ERR_INVALID_ARGUMENT;
  if (!(eps <= FLT_MAX) || !((float)eps >= FLT_MIN)) return QMUON_ERR_INVALID_ARGUMENT;
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
  L.keys.set(seed);
  L.step = (uint32_t)t;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      launch_dependent(adam_kernel(plan->state, sr, plan->per_warp), plan->n_chunks, kThreads, plan->smem, s, L);
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
