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
  depends_begin();
  if (b >= A.rows * A.per_row) return;
  int64_t row, group;
  row_and_group(A, b, &row, &group);
  float v[32];
  load_row<DT, 32>(static_cast<const unsigned char*>(A.src) + (row * A.ld + 32 * group) * elem_size(DT), 32, A.vec, v);
  A.scale_out[b] = (uint8_t)encode_row<32>(static_cast<uint8_t*>(A.dst) + 32 * b, true, A.pvec, v);
}

// Rows that start anywhere: a warp per group, kUnroll groups at a time.
constexpr int kUnroll = 8;
template <int DT>
__global__ void __launch_bounds__(kThreads) encode_lanes_kernel(Args A) {
  const int64_t total = A.rows * A.per_row;
  const int64_t b0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kUnroll;
  const int lane = threadIdx.x & 31;
  depends_begin();
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
  depends_begin();
  if (b >= A.rows * A.per_row) return;
  int64_t row, group;
  row_and_group(A, b, &row, &group);
  float v[32];
  decode_row<32>(static_cast<const uint8_t*>(A.src) + 32 * b, A.pvec, scale_of_e8m0(A.scale_in[b]), v);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = decoded<DT>(v[i]);
  store_row<DT, 32>(static_cast<unsigned char*>(A.dst) + (row * A.ld + 32 * group) * elem_size(DT), 32, A.vec, v);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) decode_lanes_kernel(Args A) {
  const int64_t total = A.rows * A.per_row;
  const int64_t b0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kUnroll;
  const int lane = threadIdx.x & 31;
  depends_begin();
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
struct RepackArgs {
  Repack job[3];
  int64_t first[3];   // the jobs' first CTAs
  int32_t n;
};
__global__ void __launch_bounds__(kThreads) repack_kernel(const __grid_constant__ RepackArgs A) {
  depends_begin();
  const int k = A.n > 2 && blockIdx.x >= A.first[2] ? 2 : A.n > 1 && blockIdx.x >= A.first[1] ? 1 : 0;
  const Repack& J = A.job[k];
  const int64_t per = (J.cols + 7) >> 3, e = ((int64_t)blockIdx.x - A.first[k]) * kThreads + threadIdx.x;
  if (e >= J.rows * per) return;
  const int64_t row = e / per, c = (e - row * per) * 8;
  const uint16_t* p = J.src + row * J.ld_src + c;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = c + 2 * i < J.cols ? p[2 * i] : 0u, b = c + 2 * i + 1 < J.cols ? p[2 * i + 1] : 0u;
    w[i] = a | (b << 16);
  }
  *reinterpret_cast<uint4*>(J.dst + row * J.ld_dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
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

cudaError_t launch_repack(const Repack* jobs, int n, cudaStream_t s) {
  RepackArgs A{};
  int64_t grid = 0;
  for (int i = 0; i < n; ++i) {
    A.job[i] = jobs[i];
    A.first[i] = grid;
    grid += ceil_div(jobs[i].rows * ((jobs[i].cols + 7) / 8), kThreads);
  }
  A.n = n;
  return n == 0 ? cudaSuccess : launch_dependent(repack_kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, A);
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
