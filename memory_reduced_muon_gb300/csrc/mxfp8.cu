// 8-bit activation checkpoints: MXFP8 carriers (E4M3 codes, one E8M0 exponent
// per 32 row elements) of any activation, and back.
//
// Both directions move each byte once and are bound by DRAM.  A thread takes
// one scale's 32 elements: its maximum needs no other thread, 16-bit values
// come and go as two whole sectors of 32 bytes, codes as one.  Rows that do
// not start on 16 bytes take a warp per 32 elements, one element per lane.
#include "qm_lm.h"

namespace qm {
namespace lm {
namespace {

constexpr int kThreads = 256;

struct Args {
  const void* src;       // encode: rows; decode: codes
  const uint8_t* scale_in;
  void* dst;             // encode: codes; decode: rows
  uint8_t* scale_out;
  int64_t rows, per_row; // per_row: groups of 32 in a row
  int64_t ld;            // of the rows, in elements
  int32_t vec, pvec;     // access classes of the rows and of the codes
};

__device__ __forceinline__ void row_and_group(const Args& A, int64_t b, int64_t* row, int64_t* group) {
  if (A.rows * A.per_row <= 0xFFFFFFFFll) {
    const uint32_t r = (uint32_t)b / (uint32_t)A.per_row;
    *row = r;
    *group = (uint32_t)b - r * (uint32_t)A.per_row;
  } else {
    *row = b / A.per_row;
    *group = b - *row * A.per_row;
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) encode_kernel(Args A) {
  const int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  depends_wait();
  if (b >= A.rows * A.per_row) return;
  int64_t row, group;
  row_and_group(A, b, &row, &group);
  float v[32];
  load_row32<DT>(static_cast<const unsigned char*>(A.src) + (row * A.ld + 32 * group) * elem_size(DT), 32, A.vec, v);
  A.scale_out[b] = (uint8_t)encode_row32(static_cast<uint8_t*>(A.dst) + 32 * b, A.pvec, v);
}

// Rows that start anywhere: a warp per group, kUnroll groups at a time.
constexpr int kUnroll = 8;
template <int DT>
__global__ void __launch_bounds__(kThreads) encode_lanes_kernel(Args A) {
  const int64_t total = A.rows * A.per_row;
  const int64_t b0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kUnroll;
  const int lane = threadIdx.x & 31;
  depends_wait();
  float v[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    v[i] = 0.0f;
    if (b0 + i < total) {
      int64_t row, group;
      row_and_group(A, b0 + i, &row, &group);
      v[i] = load_elem<DT>(A.src, row * A.ld + 32 * group + lane);
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    if (b0 + i >= total) break;
    // fmaxf ignores a NaN; not negative, so ordered as integers
    const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fabsf(v[i]), 0.0f))));
    const int byte = e8m0_of_amax(amax);
    static_cast<uint8_t*>(A.dst)[32 * (b0 + i) + lane] = (uint8_t)cvt_e4m3x2(__fmul_rn(v[i], pow2_from_e8m0(byte)), 0.0f);
    if (lane == 0) A.scale_out[b0 + i] = (uint8_t)byte;
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) decode_kernel(Args A) {
  const int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  depends_wait();
  if (b >= A.rows * A.per_row) return;
  int64_t row, group;
  row_and_group(A, b, &row, &group);
  const uint8_t* p = static_cast<const uint8_t*>(A.src) + 32 * b;
  uint32_t w[8];
  if (A.pvec == 2) {
    load32b(p, w);
  } else {
    const uint4 lo = *reinterpret_cast<const uint4*>(p), hi = *reinterpret_cast<const uint4*>(p + 16);
    w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w, w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
  }
  const float s = scale_of_e8m0(A.scale_in[b]);
  float v[32];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 a = mul2_rn(e4m3x2_to(w[i] & 0xFFFFu), s), c = mul2_rn(e4m3x2_to(w[i] >> 16), s);
    v[4 * i] = decoded<DT>(a.x), v[4 * i + 1] = decoded<DT>(a.y), v[4 * i + 2] = decoded<DT>(c.x), v[4 * i + 3] = decoded<DT>(c.y);
  }
  store_row32<DT>(static_cast<unsigned char*>(A.dst) + (row * A.ld + 32 * group) * elem_size(DT), 32, A.vec, v);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) decode_lanes_kernel(Args A) {
  const int64_t total = A.rows * A.per_row;
  const int64_t b0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kUnroll;
  const int lane = threadIdx.x & 31;
  depends_wait();
  uint32_t code[kUnroll], byte[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    code[i] = byte[i] = 0;
    if (b0 + i < total) {
      code[i] = static_cast<const uint8_t*>(A.src)[32 * (b0 + i) + lane];
      byte[i] = A.scale_in[b0 + i];
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    if (b0 + i >= total) break;
    int64_t row, group;
    row_and_group(A, b0 + i, &row, &group);
    store_elem<DT>(A.dst, row * A.ld + 32 * group + lane, decoded<DT>(__fmul_rn(e4m3x2_to(code[i]).x, scale_of_e8m0(byte[i]))));
  }
}

// Rows of 16-bit elements to rows that start on 16 bytes: eight elements per
// thread, written as one vector; the elements behind the last are left as they
// are (the tensor maps that read the copy end at the last column).
__global__ void __launch_bounds__(kThreads) repack_kernel(const uint16_t* src, int64_t ld_src, uint16_t* dst, int64_t ld_dst,
                                                          int64_t rows, int64_t cols) {
  const int64_t per = (cols + 7) >> 3, e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  depends_wait();
  if (e >= rows * per) return;
  const int64_t row = e / per, c = (e - row * per) * 8;
  const uint16_t* p = src + row * ld_src + c;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = c + 2 * i < cols ? p[2 * i] : 0u, b = c + 2 * i + 1 < cols ? p[2 * i + 1] : 0u;
    w[i] = a | (b << 16);
  }
  *reinterpret_cast<uint4*>(dst + row * ld_dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <class K>
cudaError_t launch_groups(K kernel, const Args& A, bool lanes, cudaStream_t s) {
  const int64_t groups = A.rows * A.per_row;
  const int64_t grid = ceil_div(groups, lanes ? kThreads / 32 * kUnroll : kThreads);
  return launch_dependent(kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, A);
}

bool check(const qmuon_mxfp8* c, qmuon_status* st) {
  *st = QMUON_ERR_INVALID_ARGUMENT;
  if (!c || c->rows < 0 || c->cols < 1 || c->cols > ((int64_t)1 << 30) || c->rows > ((int64_t)1 << 40) / c->cols) return false;
  if (c->dtype < QMUON_BF16 || c->dtype > QMUON_FP32) return false;
  if (c->cols % QMUON_SCALE_BLOCK) return *st = QMUON_ERR_UNSUPPORTED, false;
  if (c->rows == 0) return *st = QMUON_OK, false;
  if (!c->x || !c->payload || !c->scale_inv || c->ld_x < c->cols || c->ld_x > ((int64_t)1 << 40)) return false;
  if (!is_aligned(c->x, elem_size(c->dtype)) || !is_aligned(c->payload, 16)) return false;
  // the grid's limit: 2^31 - 1 CTAs of 256 groups, or of 64
  if (c->rows * (c->cols / 32) > ((int64_t)1 << 31) * 63) return *st = QMUON_ERR_UNSUPPORTED, false;
  return true;
}

}  // namespace

cudaError_t launch_decode(const uint8_t* payload, const uint8_t* scale, void* x, int64_t rows, int64_t cols, int64_t ld, int dt,
                          cudaStream_t s) {
  const Args A{payload, scale, x, nullptr, rows, cols / 32, ld, vec_class(x, ld, elem_size(dt)), vec_class(payload, 32, 1)};
  const bool lanes = A.vec == 0;
  auto pick = [&](auto whole, auto by_lane) { return launch_groups(lanes ? by_lane : whole, A, lanes, s); };
  if (dt == QMUON_BF16) return pick(decode_kernel<QMUON_BF16>, decode_lanes_kernel<QMUON_BF16>);
  if (dt == QMUON_FP16) return pick(decode_kernel<QMUON_FP16>, decode_lanes_kernel<QMUON_FP16>);
  return pick(decode_kernel<QMUON_FP32>, decode_lanes_kernel<QMUON_FP32>);
}

cudaError_t launch_repack(const void* src, int64_t ld_src, void* dst, int64_t ld_dst, int64_t rows, int64_t cols, cudaStream_t s) {
  const int64_t grid = ceil_div(rows * ((cols + 7) / 8), kThreads);
  return launch_dependent(repack_kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, src, ld_src, dst, ld_dst, rows, cols);
}

}  // namespace lm
}  // namespace qm

using namespace qm;

extern "C" qmuon_status qmuon_mxfp8_encode(const qmuon_mxfp8* c, void* stream) {
  NvtxRange nvtx_range("qmuon_mxfp8_encode");
  return no_throw("qmuon_mxfp8_encode", [&]() -> qmuon_status {
    qmuon_status st;
    if (!lm::check(c, &st)) return st;
    const lm::Args A{c->x,    nullptr,           c->payload, c->scale_inv,
                     c->rows, c->cols / 32,      c->ld_x,    lm::vec_class(c->x, c->ld_x, elem_size(c->dtype)),
                     lm::vec_class(c->payload, 32, 1)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool lanes = A.vec == 0;
    auto pick = [&](auto whole, auto by_lane) { return lm::launch_groups(lanes ? by_lane : whole, A, lanes, s); };
    const cudaError_t e = c->dtype == QMUON_BF16   ? pick(lm::encode_kernel<QMUON_BF16>, lm::encode_lanes_kernel<QMUON_BF16>)
                          : c->dtype == QMUON_FP16 ? pick(lm::encode_kernel<QMUON_FP16>, lm::encode_lanes_kernel<QMUON_FP16>)
                                                   : pick(lm::encode_kernel<QMUON_FP32>, lm::encode_lanes_kernel<QMUON_FP32>);
    return e == cudaSuccess ? QMUON_OK : set_error("qmuon_mxfp8_encode (launch)", e);
  });
}

extern "C" qmuon_status qmuon_mxfp8_decode(const qmuon_mxfp8* c, void* stream) {
  NvtxRange nvtx_range("qmuon_mxfp8_decode");
  return no_throw("qmuon_mxfp8_decode", [&]() -> qmuon_status {
    qmuon_status st;
    if (!lm::check(c, &st)) return st;
    const cudaError_t e =
        lm::launch_decode(c->payload, c->scale_inv, c->x, c->rows, c->cols, c->ld_x, c->dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? QMUON_OK : set_error("qmuon_mxfp8_decode (launch)", e);
  });
}
