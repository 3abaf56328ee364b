// Token embedding: lookup with scaling, and its gradient by sorted tokens.
//
//   out[t] = scale table[tokens[t]]            (zeros for a token outside [0, vocab))
//   dtable[v] = scale sum over t with tokens[t] = v of dout[t]
//
// The lookup moves each row once; the gradient reads dout once and writes every
// row of dtable once.  Both are bound by DRAM.
//
// The gradient's order is fixed: tokens are sorted stably (radix passes of up
// to 9 bits), so that each row's terms lie one after another in ascending t,
// and are added in fp32 in that order, kPiece positions at a time.  A piece
// whose run of a token neither begins before it nor goes on behind it writes
// its row itself; runs that cross pieces leave fp32 partial sums, which a second
// kernel adds: warp w those of the run's pieces w, w + 8, ..., then the warps'
// sums.  No atomics touch a result.
#include <algorithm>

#include "qm_lm.h"

namespace qm {
namespace lm {
namespace {

constexpr int kThreads = 256;

template <class Tok>
__device__ __forceinline__ int64_t token_at(const void* tokens, int64_t t) {
  return (int64_t) static_cast<const Tok*>(tokens)[t];
}

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
struct LookupArgs {
  const void* table;
  const void* tokens;
  void* out;
  int64_t n, vocab, ld_table, ld_out;
  int32_t cols, bits64;
  float scale;
};

// VEC: rows of 16-byte vectors, else single elements.  A row belongs to blockDim.x threads, blockDim.y rows to a CTA.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) lookup_kernel(LookupArgs A) {
  constexpr int es = elem_size(DT), K = VEC ? 16 / es : 1;
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  depends_begin();
  if (t >= A.n) return;
  const int64_t v = A.bits64 ? token_at<int64_t>(A.tokens, t) : token_at<int32_t>(A.tokens, t);
  const bool there = v >= 0 && v < A.vocab;
  const unsigned char* src = static_cast<const unsigned char*>(A.table) + (there ? v : 0) * A.ld_table * es;
  unsigned char* dst = static_cast<unsigned char*>(A.out) + t * A.ld_out * es;
  const int n = A.cols / K, step = blockDim.x * gridDim.y;
  constexpr int U = VEC ? 4 : 8;
  for (int i0 = blockIdx.y * blockDim.x + threadIdx.x; i0 < n; i0 += U * step) {
    if constexpr (VEC) {
      uint4 w[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * step;
        w[j] = make_uint4(0u, 0u, 0u, 0u);
        if (i < n && there) w[j] = *reinterpret_cast<const uint4*>(src + 16 * (int64_t)i);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * step;
        if (i >= n) break;
        float2 f[Vec16<DT>::kPairs];
        Vec16<DT>::unpack(w[j], f);
#pragma unroll
        for (int k = 0; k < Vec16<DT>::kPairs; ++k) f[k] = there ? mul2_rn(f[k], A.scale) : make_float2(0.0f, 0.0f);
        *reinterpret_cast<uint4*>(dst + 16 * (int64_t)i) = Vec16<DT>::pack(f);
      }
    } else {
      float f[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * step;
        f[j] = i < n && there ? load_elem<DT>(src, i) : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * step;
        if (i < n) store_elem<DT>(dst, i, there ? __fmul_rn(f[j], A.scale) : 0.0f);
      }
    }
  }
}

// Threads of a row, in x, and rows of a CTA, in y: up to `each` items per thread.
dim3 row_block(int64_t items, int each) {
  int x = 32;
  while (x < kThreads && (int64_t)x * each < items) x *= 2;
  return dim3(x, kThreads / x);
}

template <int DT>
cudaError_t launch_lookup(const LookupArgs& A, int sms, cudaStream_t s) {
  const bool vec = vec_class(A.table, A.ld_table, elem_size(DT)) && vec_class(A.out, A.ld_out, elem_size(DT)) &&
                   A.cols * elem_size(DT) % 16 == 0;
  const int64_t items = vec ? A.cols * elem_size(DT) / 16 : A.cols;
  const dim3 block = row_block(items, vec ? 4 : 8);
  const int64_t rows = ceil_div(A.n, block.y);
  // few rows: several CTAs to each, so that one token's row is not one SM's work
  const int64_t most = ceil_div(items, block.x);
  const unsigned parts = (unsigned)std::max<int64_t>(1, std::min<int64_t>(most, sms / rows));
  const dim3 grid((unsigned)rows, parts);
  return vec ? launch_dependent(lookup_kernel<DT, true>, grid, block, 0, s, A)
             : launch_dependent(lookup_kernel<DT, false>, grid, block, 0, s, A);
}

// ---------------------------------------------------------------------------
// sorting
// ---------------------------------------------------------------------------
// Keys are tokens, `vocab` standing for every token outside; a key's bits are
// sorted from the low ones up, up to 9 a pass.  A CTA takes kSortKeys keys at
// most, its warps equal shares in rounds of 32, so that a warp's keys are ranked
// in order: lanes of equal digits find one another by match, the lowest of them
// adds their number to the warp's count.
//
// Up to 8 such CTAs are one cluster, whose barriers part the passes: one launch
// sorts 65536 tokens.  That takes a few SMs 10 to 20 us, in which the others
// write zeros to the table's last rows, those of tokens too.  More tokens take
// three kernels a pass (the CTAs' counts, their sums, the moves).
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32, kRounds = 16, kSortKeys = kSortThreads * kRounds;
constexpr int kSortCluster = 8, kClusterKeys = kSortWarps * 64;   // a CTA's keys before the cluster grows
// Of the table's last rows, written meanwhile: what a few SMs' sorting time has room for.  In us, of bf16 with 16384 tokens,
// none / 16 / 32 / 64 / 96 / 128 MB: 102400 x 4096 177 / 177 / 175 / 171 / 174 / 177, 50000 x 1000 56 / 55 / 55 / 52 / 58 / 58,
// 400000 x 64 52 / 44 / 38 / 36 / 36 / 36; 65536 tokens, 102400 x 1024 121 / 122 / 122 / 121 / 120 / 118.
constexpr int64_t kFillBytes = (int64_t)64 << 20;
static_assert(kSortThreads == kDigits, "a thread per digit");

struct SortArgs {
  const void* tokens;    // first pass, or null
  const uint2* in;       // (key, position) pairs of the pass before, or null
  uint2* out;
  uint32_t* counts;      // [kDigits][CTAs]: the CTAs' digits
  int64_t n, vocab;
  int32_t bits64, shift, n_cta;
  int32_t share;         // keys of a warp, a multiple of 32
  int32_t passes;        // cluster_sort_kernel
  uint2* pairs[2];       // cluster_sort_kernel: where odd and even passes leave the pairs
  // cluster_sort_kernel, CTAs behind the first cluster: zeros to the last `fill` rows of the table's gradient
  unsigned char* table;
  int64_t fill, ld_bytes;
  int32_t vecs, across;  // of 16 bytes in a row; threads of a row, a power of two up to a CTA's
};

__device__ __forceinline__ uint2 key_of(const SortArgs& A, int64_t i) {
  if (A.in) return __ldcg(A.in + i);   // another SM's, moments ago
  const int64_t v = A.bits64 ? token_at<int64_t>(A.tokens, i) : token_at<int32_t>(A.tokens, i);
  return make_uint2(v >= 0 && v < A.vocab ? (uint32_t)v : (uint32_t)A.vocab, (uint32_t)i);
}

// The keys of a warp, and the rank of each among the warp's keys of its digit; `count` is the warp's number of each digit.
struct WarpKeys {
  uint2 kv[kRounds];
  uint32_t rank[kRounds];
};
__device__ __forceinline__ void rank_keys(const SortArgs& A, int64_t first, int lane, WarpKeys& K, uint16_t* count) {
  const int64_t end = first + A.share < A.n ? first + A.share : A.n;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = first + r * 32 + lane;
    K.kv[r] = i < end ? key_of(A, i) : make_uint2(0u, 0u);
  }
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    if (first + r * 32 >= end) break;   // the same for all lanes
    const bool valid = first + r * 32 + lane < end;
    const uint32_t digit = valid ? (K.kv[r].x >> A.shift) & (kDigits - 1) : (uint32_t)kDigits;
    const uint32_t peers = __match_any_sync(0xffffffffu, digit);
    const uint32_t below = __popc(peers & ((1u << lane) - 1u));
    uint32_t old = 0;
    if (valid) old = count[digit];
    __syncwarp();
    if (valid && below == 0) count[digit] = (uint16_t)(old + __popc(peers));
    __syncwarp();
    K.rank[r] = old + below;
  }
}
__device__ __forceinline__ void move_keys(const SortArgs& A, int64_t first, int lane, const WarpKeys& K, const uint16_t* before,
                                          const uint32_t* base, uint2* out) {
  const int64_t end = first + A.share < A.n ? first + A.share : A.n;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    if (first + r * 32 + lane < end) {
      const uint32_t digit = (K.kv[r].x >> A.shift) & (kDigits - 1);
      out[base[digit] + before[digit] + K.rank[r]] = K.kv[r];
    }
  }
}
// Thread d: the CTA's number of digit d; count[w][d] becomes the number in the warps before w.
__device__ __forceinline__ uint32_t warps_before(uint16_t (*count)[kDigits]) {
  uint32_t sum = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    const uint32_t k = count[w][threadIdx.x];
    count[w][threadIdx.x] = (uint16_t)sum;
    sum += k;
  }
  return sum;
}
// Exclusive sum of v over the CTA's 512 threads.
__device__ __forceinline__ uint32_t sum_before(uint32_t v, uint32_t* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  const uint32_t w = lane < warp ? warp_sum[lane] : 0u;   // the warps before
  return incl - v + __reduce_add_sync(0xffffffffu, w);
}
// Every write of the cluster's CTAs before it is seen by all of them behind it.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kSortThreads) cluster_sort_kernel(SortArgs A) {
  __shared__ uint16_t count[kSortWarps][kDigits];
  __shared__ uint32_t base[kDigits], warp_sum[kSortWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = threadIdx.x;
  const int64_t first = ((int64_t)blockIdx.x * kSortWarps + warp) * A.share;
  depends_begin();
  if ((int)blockIdx.x >= A.n_cta) {
    // rows of less than a CTA's vectors share it (one row at a time, 400000 x 64 bf16 took 738 us, 50000 x 1000 96)
    const int down = kSortThreads / A.across;
    const int64_t step = (int64_t)(gridDim.x - A.n_cta) * down;
    for (int64_t r = A.vocab - A.fill + (int64_t)(blockIdx.x - A.n_cta) * down + d / A.across; r < A.vocab; r += step)
      for (int i = d & (A.across - 1); i < A.vecs; i += A.across) *reinterpret_cast<uint4*>(A.table + r * A.ld_bytes + 16 * (int64_t)i) = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  for (int pass = 0; pass < A.passes; ++pass) {
    for (int w = 0; w < kSortWarps; ++w) count[w][d] = 0;
    __syncthreads();
    WarpKeys K;
    rank_keys(A, first, lane, K, count[warp]);
    __syncthreads();
    A.counts[(int64_t)d * A.n_cta + blockIdx.x] = warps_before(count);
    cluster_barrier();
    uint32_t total = 0, mine = 0;
    uint32_t of[kSortCluster];   // all loads at once
#pragma unroll
    for (int c = 0; c < kSortCluster; ++c) of[c] = c < A.n_cta ? __ldcg(A.counts + (int64_t)d * A.n_cta + c) : 0u;
#pragma unroll
    for (int c = 0; c < kSortCluster; ++c) {
      if (c == (int)blockIdx.x) mine = total;
      total += of[c];
    }
    base[d] = sum_before(total, warp_sum) + mine;
    __syncthreads();
    move_keys(A, first, lane, K, count[warp], base, A.pairs[pass & 1]);
    cluster_barrier();
    A.in = A.pairs[pass & 1];
    A.shift += kDigitBits;
  }
}

__global__ void __launch_bounds__(kSortThreads) count_kernel(SortArgs A) {
  __shared__ uint32_t count[kDigits];
  count[threadIdx.x] = 0;
  __syncthreads();
  depends_begin();
  const int64_t base = (int64_t)blockIdx.x * kSortKeys;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * kSortThreads + threadIdx.x;
    if (i < A.n) atomicAdd(&count[(key_of(A, i).x >> A.shift) & (kDigits - 1)], 1u);
  }
  __syncthreads();
  A.counts[(int64_t)threadIdx.x * A.n_cta + blockIdx.x] = count[threadIdx.x];
}

// Where each CTA's keys of each digit go: an exclusive sum over digits, then CTAs.  One CTA; a thread per digit.
__global__ void __launch_bounds__(kDigits) offsets_kernel(uint32_t* counts, int n_cta) {
  __shared__ uint32_t warp_sum[kDigits / 32];
  depends_begin();
  uint32_t* mine = counts + (int64_t)threadIdx.x * n_cta;
  uint32_t total = 0;
#pragma unroll 8
  for (int c = 0; c < n_cta; ++c) total += mine[c];
  uint32_t at = sum_before(total, warp_sum);
#pragma unroll 8
  for (int c = 0; c < n_cta; ++c) {
    const uint32_t k = mine[c];
    mine[c] = at;
    at += k;
  }
}

__global__ void __launch_bounds__(kSortThreads) scatter_kernel(SortArgs A) {
  __shared__ uint16_t count[kSortWarps][kDigits];
  __shared__ uint32_t base[kDigits];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int w = 0; w < kSortWarps; ++w) count[w][threadIdx.x] = 0;
  __syncthreads();
  depends_begin();
  base[threadIdx.x] = A.counts[(int64_t)threadIdx.x * A.n_cta + blockIdx.x];
  const int64_t first = ((int64_t)blockIdx.x * kSortWarps + warp) * A.share;
  WarpKeys K;
  rank_keys(A, first, lane, K, count[warp]);
  __syncthreads();
  warps_before(count);
  __syncthreads();
  move_keys(A, first, lane, K, count[warp], base, A.out);
}

// ---------------------------------------------------------------------------
// sums
// ---------------------------------------------------------------------------
constexpr int kPiece = 32;    // sorted positions of a piece
constexpr int kZeros = 16;    // rows of a CTA that looks for rows without a token (102400 x 4096 bf16 166 us; 8 rows 173, 32 168)

struct SumArgs {
  const uint2* sorted;
  const void* dout;
  void* dtable;
  float* partial;        // [pieces][2][ldp]: a run that began before the piece, and one that goes on behind it
  int64_t n, vocab, ld_dout, ld_dtable, ldp;
  int64_t zero_rows;     // rows [0, zero_rows) of which those without a token become zero here
  int32_t cols, pieces, accumulate;
  float scale;
};

// N columns of a row as fp32, and back: 16-byte vectors (of the 16-bit type, or of fp32) or single elements.
template <int DT, int N>
__device__ __forceinline__ void load_cols(const void* base, int64_t e, float (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = load_elem<DT>(base, e);
  } else {
#pragma unroll
    for (int h = 0; h < N * elem_size(DT) / 16; ++h) {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(base) + e * elem_size(DT) + 16 * h);
      float2 f[Vec16<DT>::kPairs];
      Vec16<DT>::unpack(w, f);
#pragma unroll
      for (int k = 0; k < Vec16<DT>::kPairs; ++k) {
        v[h * Vec16<DT>::kElems + 2 * k] = f[k].x;
        v[h * Vec16<DT>::kElems + 2 * k + 1] = f[k].y;
      }
    }
  }
}
template <int DT, int N>
__device__ __forceinline__ void store_cols(void* base, int64_t e, const float (&v)[N]) {
  if constexpr (N == 1) {
    store_elem<DT>(base, e, v[0]);
  } else {
#pragma unroll
    for (int h = 0; h < N * elem_size(DT) / 16; ++h) {
      float2 f[Vec16<DT>::kPairs];
#pragma unroll
      for (int k = 0; k < Vec16<DT>::kPairs; ++k)
        f[k] = make_float2(v[h * Vec16<DT>::kElems + 2 * k], v[h * Vec16<DT>::kElems + 2 * k + 1]);
      *reinterpret_cast<uint4*>(static_cast<unsigned char*>(base) + e * elem_size(DT) + 16 * h) = Vec16<DT>::pack(f);
    }
  }
}

template <int GT, int N>
__device__ __forceinline__ void write_row(const SumArgs& A, int64_t row, int64_t col, const float (&sum)[N]) {
  const int64_t e = row * A.ld_dtable + col;
  float v[N];
  if (A.accumulate) {
    load_cols<GT, N>(A.dtable, e, v);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = fmaf(A.scale, sum[k], v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __fmul_rn(A.scale, sum[k]);
  }
  store_cols<GT, N>(A.dtable, e, v);
}

// The first sorted position in [lo, hi) whose key is not below `key`, or hi, by a whole warp.
__device__ __forceinline__ int64_t first_at_least(const uint2* sorted, int64_t lo, int64_t hi, uint32_t key, int lane) {
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step - 1;
    const uint32_t less = __ballot_sync(0xffffffffu, i < hi && sorted[i].x < key);   // ascending: a run of low lanes
    const int k = __popc(less);
    const int64_t next = lo + (k + 1) * step - 1;
    lo += k * step;
    if (next < hi) hi = next;
  }
  return lo;
}

// CTA (piece, slab of columns): a thread's N columns over the piece's positions; behind the pieces, CTAs that write the
// zeros of the rows without a token.
template <int DT, int GT, int N>
__global__ void __launch_bounds__(kThreads, 4) sum_kernel(SumArgs A) {
  const int64_t col = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * N;
  depends_begin();
  __shared__ int64_t range[2];
  __shared__ uint8_t there[kZeros];
  const int64_t piece = blockIdx.x;
  if (piece >= A.pieces) {
    float zero[N];
#pragma unroll
    for (int k = 0; k < N; ++k) zero[k] = 0.0f;
    const int64_t r0 = (piece - A.pieces) * kZeros;
    const int rows = (int)(A.zero_rows - r0 < kZeros ? A.zero_rows - r0 : kZeros);
    if (threadIdx.x < 64) {   // the positions of these rows' tokens
      const int warp = threadIdx.x >> 5;
      const int64_t at = first_at_least(A.sorted, 0, A.n, (uint32_t)(r0 + (warp ? rows : 0)), threadIdx.x & 31);
      if ((threadIdx.x & 31) == 0) range[warp] = at;
      if (threadIdx.x < kZeros) there[threadIdx.x] = 0;
    }
    __syncthreads();
    if (range[1] - range[0] <= (int64_t)kZeros * blockDim.x) {
      for (int64_t i = range[0] + threadIdx.x; i < range[1]; i += blockDim.x) there[A.sorted[i].x - (uint32_t)r0] = 1;
    } else {   // frequent tokens: a search per row, whose work does not grow with their number (2^20 tokens, 95% of them one,
               // 102400 x 64 bf16 3.45 -> 1.81 ms)
      for (int r = threadIdx.x >> 5; r < rows; r += blockDim.x >> 5) {
        const uint32_t key = (uint32_t)(r0 + r);
        const int64_t at = first_at_least(A.sorted, range[0], range[1], key, threadIdx.x & 31);
        if ((threadIdx.x & 31) == 0 && at < range[1]) there[r] = A.sorted[at].x == key;
      }
    }
    __syncthreads();
    if (col >= A.cols) return;
#pragma unroll 4
    for (int r = 0; r < rows; ++r)
      if (!there[r]) store_cols<GT, N>(A.dtable, (r0 + r) * A.ld_dtable + col, zero);
    return;
  }
  __shared__ uint2 mine[kPiece + 2];   // the neighbours' keys at both ends
  const int64_t i0 = piece * kPiece;
  const int n = (int)(A.n - i0 < kPiece ? A.n - i0 : kPiece);
  if (threadIdx.x < n + 2) {
    const int64_t i = i0 - 1 + threadIdx.x;
    mine[threadIdx.x] = i >= 0 && i < A.n ? A.sorted[i] : make_uint2(0xFFFFFFFFu, 0u);
  }
  __syncthreads();
  if (col >= A.cols) return;
  float sum[N];
#pragma unroll
  for (int k = 0; k < N; ++k) sum[k] = 0.0f;
  bool before = mine[0].x == mine[1].x;   // the run began in an earlier piece
  constexpr int U = N == 1 ? 16 : 4;      // rows in flight (single columns: 4 rows 195 us, 16 180, for 65536 x 1001 fp32)
  for (int j0 = 0; j0 < n; j0 += U) {
    float v[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j0 + u < n && mine[j0 + u + 1].x < (uint32_t)A.vocab) {
        load_cols<DT, N>(A.dout, (int64_t)mine[j0 + u + 1].y * A.ld_dout + col, v[u]);
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) v[u][k] = 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u;
      if (j >= n) break;
      const uint32_t key = mine[j + 1].x;
#pragma unroll
      for (int k = 0; k < N; ++k) sum[k] += v[u][k];
      const bool ends = mine[j + 2].x != key;
      if (!ends && j + 1 < n) continue;
      if (key < (uint32_t)A.vocab) {
        if (!before && ends) {
          write_row<GT, N>(A, key, col, sum);
        } else {
          // slot 0: the run began before this piece (and may go on); slot 1: it begins here and goes on
          float* p = A.partial + (piece * 2 + (before ? 0 : 1)) * A.ldp + col;
          store_cols<QMUON_FP32, N>(p, 0, sum);
        }
      }
#pragma unroll
      for (int k = 0; k < N; ++k) sum[k] = 0.0f;
      before = false;
    }
  }
}

// The runs that cross pieces: CTA (piece, slab) adds up the run that begins in its piece and goes on behind it.  Warp w
// takes the run's pieces w, w + 8, ... in order, 4 at a time on their way, and the warps' sums are added in order: a token
// that is most of a batch has thousands of pieces.
constexpr int kJoinWarps = 8;
template <int GT, int N>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(SumArgs A) {
  __shared__ float sums[kJoinWarps][32][N];
  const int warp = threadIdx.y;
  depends_begin();
  const int64_t p = blockIdx.x, last = (p + 1) * kPiece - 1;   // not the last piece: last + 1 is a position
  // all at once: one way to L2
  const uint32_t key = A.sorted[last].x, behind = A.sorted[last + 1].x, first = A.sorted[p * kPiece].x;
  const uint32_t ahead = p > 0 ? A.sorted[p * kPiece - 1].x : 0xFFFFFFFFu;
  const uint32_t next = p + 2 < A.pieces ? A.sorted[(p + 2) * kPiece].x : 0xFFFFFFFFu;
  if (key >= (uint32_t)A.vocab || behind != key) return;
  if (first == key && ahead == key) return;   // it began before
  // the first piece behind it that begins with another key: most runs end in the next one, so the search starts there
  int64_t lo = p + 2, hi = p + 2, step = 1;
  if (next == key)
    do lo = ++hi, hi += step, step *= 2;
    while (hi < A.pieces && A.sorted[hi * kPiece].x == key);
  if (hi > A.pieces) hi = A.pieces;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (A.sorted[mid * kPiece].x == key) lo = mid + 1;
    else hi = mid;
  }
  for (int64_t slab = (int64_t)blockIdx.y * 32 * N; slab < A.cols; slab += (int64_t)gridDim.y * 32 * N) {
    const int64_t col = slab + threadIdx.x * N;
    const bool there = col < A.cols;
    float sum[N];
#pragma unroll
    for (int k = 0; k < N; ++k) sum[k] = 0.0f;
    if (there) {
      if (warp == 0) load_cols<QMUON_FP32, N>(A.partial, (p * 2 + 1) * A.ldp + col, sum);
      for (int64_t j = p + 1 + warp; j < lo; j += 4 * kJoinWarps) {
        float v[4][N];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (j + c * kJoinWarps < lo) {
            load_cols<QMUON_FP32, N>(A.partial, (j + c * kJoinWarps) * 2 * A.ldp + col, v[c]);
          } else {
#pragma unroll
            for (int k = 0; k < N; ++k) v[c][k] = 0.0f;
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int k = 0; k < N; ++k) sum[k] += v[c][k];
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) sums[warp][threadIdx.x][k] = sum[k];
    __syncthreads();
    if (warp == 0 && there) {
#pragma unroll
      for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
        for (int k = 0; k < N; ++k) sum[k] += sums[w][threadIdx.x][k];
      write_row<GT, N>(A, key, col, sum);
    }
    __syncthreads();
  }
}

struct Layout {
  int passes, n_cta, pieces;
  size_t pairs[2], counts, partial, total;
  int64_t ldp;
};

Layout layout_of(int64_t n, int64_t vocab, int64_t cols) {
  Layout L{};
  L.passes = 1;
  while (L.passes * kDigitBits < 32 && (vocab >> (L.passes * kDigitBits)) != 0) ++L.passes;   // keys 0 .. vocab
  L.n_cta = (int)std::max(std::min(ceil_div(n, kClusterKeys), (int64_t)kSortCluster), ceil_div(n, kSortKeys));
  L.pieces = (int)ceil_div(n, kPiece);
  L.ldp = (int64_t)round_up((size_t)cols, 8);
  size_t at = 0;
  for (size_t& p : L.pairs) p = at, at += round_up((size_t)n * 8, 256);
  L.counts = at, at += round_up((size_t)kDigits * L.n_cta * 4, 256);
  L.partial = at, at += round_up((size_t)L.pieces * 2 * L.ldp * 4, 256);
  L.total = std::max<size_t>(at, 256);   // no tokens: 0 would be a refusal
  return L;
}

constexpr int64_t kMaxTokens = (int64_t)1 << 28, kMaxVocab = ((int64_t)1 << 31) - 2, kMaxCols = (int64_t)1 << 22;

bool sizes_ok(int64_t n, int64_t vocab, int64_t cols) {
  return n >= 0 && n <= kMaxTokens && vocab >= 1 && vocab <= kMaxVocab && cols >= 1 && cols <= kMaxCols &&
         vocab <= ((int64_t)1 << 40) / cols;
}
bool rows_ok(const void* p, int64_t ld, int64_t cols, int es) {
  return p && is_aligned(p, es) && ld >= cols && ld <= ((int64_t)1 << 40);
}
bool is_type(int dt) { return dt == QMUON_BF16 || dt == QMUON_FP16 || dt == QMUON_FP32; }
bool tokens_ok(const void* p, int bits) { return p && (bits == 32 || bits == 64) && is_aligned(p, bits / 8); }

cudaError_t launch_cluster(const SortArgs& A, int sms, cudaStream_t s) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = A.n_cta;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(A.fill ? std::max(2, sms / A.n_cta) * A.n_cta : A.n_cta);   // whole clusters
  cfg.blockDim = dim3(kSortThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, cluster_sort_kernel, A);
}

template <int DT, int GT, int N>
cudaError_t launch_sums(const SumArgs& A, cudaStream_t s) {
  const unsigned slabs = (unsigned)ceil_div(A.cols, (int64_t)kThreads * N);
  const int64_t zeros = ceil_div(A.zero_rows, kZeros);
  const int threads = (int)std::min<int64_t>(kThreads, round_up((size_t)ceil_div(A.cols, N), 32));
  cudaError_t e = launch_dependent(sum_kernel<DT, GT, N>, dim3((unsigned)(A.pieces + zeros), slabs), dim3(std::max(threads, 64)), 0, s, A);
  if (e == cudaSuccess && A.pieces > 1)
    e = launch_dependent(join_kernel<GT, N>, dim3(A.pieces - 1, (unsigned)std::min<int64_t>(ceil_div(A.cols, (int64_t)32 * N), 4096)), dim3(32, kJoinWarps), 0, s, A);
  return e;
}
template <int DT>
cudaError_t launch_sums_of(const SumArgs& A, int gt, cudaStream_t s) {
  const int gs = elem_size(gt);
  constexpr int K = 16 / elem_size(DT);
  const bool vec = A.cols % K == 0 && vec_class(A.dout, A.ld_dout, elem_size(DT)) && vec_class(A.dtable, A.ld_dtable, gs);
  if (gt == QMUON_FP32)
    return vec ? launch_sums<DT, QMUON_FP32, K>(A, s) : launch_sums<DT, QMUON_FP32, 1>(A, s);
  return vec ? launch_sums<DT, DT, K>(A, s) : launch_sums<DT, DT, 1>(A, s);
}

}  // namespace
}  // namespace lm
}  // namespace qm

using namespace qm;
using namespace qm::lm;

extern "C" qmuon_status qmuon_embedding_forward(const qmuon_embedding* c, void* stream) {
  NvtxRange nvtx_range("qmuon_embedding_forward");
  return no_throw("qmuon_embedding_forward", [&]() -> qmuon_status {
    if (!c || !sizes_ok(c->n_tokens, c->vocab, c->cols) || !is_type(c->dtype)) return QMUON_ERR_INVALID_ARGUMENT;
    if (c->n_tokens == 0) return QMUON_OK;
    const int es = elem_size(c->dtype);
    if (!tokens_ok(c->tokens, c->token_bits) || !rows_ok(c->table, c->ld_table, c->cols, es) || !rows_ok(c->out, c->ld_out, c->cols, es))
      return QMUON_ERR_INVALID_ARGUMENT;
    const int sms = num_sms();
    if (sms <= 0) return set_error_msg("qmuon_embedding_forward: SM count query failed", QMUON_ERR_CUDA);
    const LookupArgs A{c->table,  c->tokens,        c->out,                  c->n_tokens, c->vocab, c->ld_table,
                       c->ld_out, (int32_t)c->cols, c->token_bits == 64, c->scale};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = c->dtype == QMUON_BF16   ? launch_lookup<QMUON_BF16>(A, sms, s)
                          : c->dtype == QMUON_FP16 ? launch_lookup<QMUON_FP16>(A, sms, s)
                                                   : launch_lookup<QMUON_FP32>(A, sms, s);
    return e == cudaSuccess ? QMUON_OK : set_error("qmuon_embedding_forward (launch)", e);
  });
}

extern "C" size_t qmuon_embedding_workspace_size(int64_t n_tokens, int64_t vocab, int64_t cols) {
  return sizes_ok(n_tokens, vocab, cols) ? layout_of(n_tokens, vocab, cols).total : 0;
}

extern "C" qmuon_status qmuon_embedding_backward(const qmuon_embedding_grad* c, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("qmuon_embedding_backward");
  return no_throw("qmuon_embedding_backward", [&]() -> qmuon_status {
    if (!c || !sizes_ok(c->n_tokens, c->vocab, c->cols) || !is_type(c->dtype)) return QMUON_ERR_INVALID_ARGUMENT;
    if (c->grad_dtype != c->dtype && c->grad_dtype != QMUON_FP32) return QMUON_ERR_INVALID_ARGUMENT;
    const int es = elem_size(c->dtype), gs = elem_size(c->grad_dtype);
    if (!rows_ok(c->dtable, c->ld_dtable, c->cols, gs) || !ws || !is_aligned(ws, 256)) return QMUON_ERR_INVALID_ARGUMENT;
    if (c->n_tokens > 0 && (!tokens_ok(c->tokens, c->token_bits) || !rows_ok(c->dout, c->ld_dout, c->cols, es)))
      return QMUON_ERR_INVALID_ARGUMENT;
    const Layout L = layout_of(c->n_tokens, c->vocab, c->cols);
    if (ws_bytes < L.total) return QMUON_ERR_WORKSPACE_TOO_SMALL;
    if (c->n_tokens == 0 && c->accumulate) return QMUON_OK;
    unsigned char* w = static_cast<unsigned char*>(ws);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int sms = num_sms();
    if (sms <= 0) return set_error_msg("qmuon_embedding_backward: SM count query failed", QMUON_ERR_CUDA);
    cudaError_t e = cudaSuccess;
    int64_t zero_rows = c->accumulate ? 0 : c->vocab;
    const uint2* sorted = reinterpret_cast<uint2*>(w + L.pairs[(L.passes - 1) & 1]);
    if (c->n_tokens > 0) {
      SortArgs A{};
      A.tokens = c->tokens;
      A.counts = reinterpret_cast<uint32_t*>(w + L.counts);
      A.n = c->n_tokens, A.vocab = c->vocab, A.bits64 = c->token_bits == 64;
      A.n_cta = L.n_cta, A.passes = L.passes;
      // equal shares: the warps of the last CTA are not idle where there are few tokens
      A.share = (int32_t)round_up((size_t)ceil_div(c->n_tokens, (int64_t)L.n_cta * kSortWarps), 32);
      for (int i = 0; i < 2; ++i) A.pairs[i] = reinterpret_cast<uint2*>(w + L.pairs[i]);
      if (L.n_cta <= kSortCluster) {
        const int64_t bytes = c->cols * gs;
        if (!c->accumulate && bytes % 16 == 0 && vec_class(c->dtable, c->ld_dtable, gs)) {
          A.table = static_cast<unsigned char*>(c->dtable);
          A.fill = std::min(c->vocab, kFillBytes / bytes);
          A.ld_bytes = c->ld_dtable * gs;
          A.vecs = (int32_t)(bytes / 16);
          for (A.across = 1; A.across < A.vecs && A.across < kSortThreads;) A.across *= 2;
          zero_rows -= A.fill;
        }
        e = launch_cluster(A, sms, s);
      } else {
        A.share = kSortKeys / kSortWarps;   // as count_kernel takes them
        for (int p = 0; p < L.passes && e == cudaSuccess; ++p, A.shift += kDigitBits) {
          A.out = A.pairs[p & 1];
          e = launch_dependent(count_kernel, dim3(L.n_cta), dim3(kSortThreads), 0, s, A);
          if (e == cudaSuccess) e = launch_dependent(offsets_kernel, dim3(1), dim3(kDigits), 0, s, A.counts, L.n_cta);
          if (e == cudaSuccess) e = launch_dependent(scatter_kernel, dim3(L.n_cta), dim3(kSortThreads), 0, s, A);
          A.in = A.out;
        }
      }
    }
    if (e != cudaSuccess) return set_error("qmuon_embedding_backward (sort)", e);
    const SumArgs A{sorted, c->dout, c->dtable, reinterpret_cast<float*>(w + L.partial), c->n_tokens, c->vocab, c->ld_dout,
                    c->ld_dtable, L.ldp, zero_rows, (int32_t)c->cols, L.pieces, c->accumulate != 0, c->scale};
    e = c->dtype == QMUON_BF16   ? launch_sums_of<QMUON_BF16>(A, c->grad_dtype, s)
        : c->dtype == QMUON_FP16 ? launch_sums_of<QMUON_FP16>(A, c->grad_dtype, s)
                                 : launch_sums_of<QMUON_FP32>(A, c->grad_dtype, s);
    return e == cudaSuccess ? QMUON_OK : set_error("qmuon_embedding_backward (launch)", e);
  });
}
