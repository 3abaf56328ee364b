// Gated feed-forward block, forward and backward, on tcgen05 tensor cores.
//
//   gate = x Wg^T   up = x Wu^T   h = act(gate) up
//   dgate = dh up act'(gate)   dup = dh act(gate)
//   dx = dgate Wg + dup Wu   dWg = dgate^T x   dWu = dup^T x
//
// One kernel makes all the products.  A persistent CTA pair (cta_group::2) runs
// units of work, each a 256 x 256 accumulator over a range of K: in the forward
// product 256 rows by 128 columns of gate and the same 128 of up (one CTA of the
// pair brings the rows of Wg, the other those of Wu), so that a thread of the
// epilogue holds both and the activation, the product and the 8-bit codes need
// nothing from memory; in the gradients 256 x 256 of dx, dWg or dWu.  The
// operands are read where they lie: K-major for x W^T, MN-major for the weights
// in dx and for both operands in dW, as the instruction descriptor says.
//
// The gradients dgate and dup are rounded to the type of the activations before
// the products that read them (tensor cores take 16-bit operands of one type).
// Their roundings are independent of the result's own and as large, relative to
// its norm: in bf16 the results are off by 0.0024 instead of 0.0017.  fp16 has
// no room for small ones (dh of 1e-5 would leave a weight's gradient off by 3%
// of its norm), so there both are held times a power of two, one for the call,
// that dh's largest magnitude sets (dh_scale), and the products' sums are
// divided by it, which is exact.
//
// Few tiles: the K range is split over units, whose fp32 partial sums go
// through the workspace and a second kernel that adds them in order.  Few rows,
// and small products, go through the cores' registers (few_kernel).
//
// On one GB300, 8192 x 4096 x 14336 bf16: the tensor pipe is busy 94% (forward)
// and 97% (gradients) of the time, 513 cycles per K block of 64 out of 512, and
// the power cap sets the clock (1.65 GHz): forward to 8-bit checkpoints 0.96 to
// 1.15 ms (2.0 to 1.67 PFLOP/s), the products of the backward pass 1.9 to 2.2.
// The tensor cores cut their fp32 sums where fp32 would round: sums over K come
// out smaller by 1e-9 K of their magnitude (the library's too).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <type_traits>

#include "qm_lm.h"
#include "qm_tc.h"

namespace qm {
namespace lm {
namespace {

using namespace tc;

constexpr int kTile = 256, kBK = 64;
constexpr int kEpiWarps = 8;                       // two per TMEM lane quarter
constexpr int kThreads = 64 + 32 * kEpiWarps;      // warp 0 TMA, warp 1 MMA, warps 2.. epilogue
constexpr int kStages = 7;
constexpr uint32_t kStageBytes = 4 * kBox;         // per CTA: 128 x 64 of A, 128 x 64 of B
constexpr uint32_t kTmemCols = 512;                // two accumulators of 256 columns
constexpr size_t kSmem = (size_t)kStages * kStageBytes + 1024 + 256;
static_assert(kWsHeader == 64 * 4, "clear_kernel's threads");
static_assert(kSmem <= 232448, "dynamic shared memory above the 227 KB a CTA may use");

enum { K_FWD = 0, K_BWD = 1, K_GRAD = 2 };
// Tile rows that run side by side: what the pairs read at a time is these rows' operand and as many columns' as there are
// pairs left.  8192 x 4096 x 14336: forward 8 rows 964 us, 16 955, 32 1044, 4 998; gradients 2205, 2270, 2370, 2230.
__host__ __device__ constexpr int group_rows(int kind) { return kind == K_GRAD ? 8 : 16; }

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------
// The logistic function; 0 and 1 at the ends, NaN for NaN.  Already 0 from -87.4 down, where the quotient's divisor passes
// 2^126 and the true value 1.2e-38: silu and its slope lack 1e-36 there.
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

template <int ACT>
__device__ __forceinline__ float act_of(float g) {
  if constexpr (ACT == QMUON_ACT_SILU) {
    return g * logistic(g);
  } else if constexpr (ACT == QMUON_ACT_GELU) {
    return g * (0.5f * erfcf(g * -0.70710678f));
  } else {   // 0.5 (1 + tanh z) = logistic(2 z), z = sqrt(2 / pi) (g + 0.044715 g^3)
    return g * logistic(1.5957691f * g * fmaf(0.044715f * g, g, 1.0f));
  }
}
// The activation and its derivative.
template <int ACT>
__device__ __forceinline__ float2 act_and_slope(float g) {
  if constexpr (ACT == QMUON_ACT_SILU) {
    const float s = logistic(g);
    return make_float2(g * s, s * fmaf(g, 1.0f - s, 1.0f));
  } else if constexpr (ACT == QMUON_ACT_GELU) {
    const float cdf = 0.5f * erfcf(g * -0.70710678f);
    return make_float2(g * cdf, fmaf(g, 0.39894228f * __expf(-0.5f * g * g), cdf));
  } else {
    const float s = logistic(1.5957691f * g * fmaf(0.044715f * g, g, 1.0f));
    // beyond +-16 the slope is 0 or 1 in fp32; there the polynomial may overflow where s (1 - s) is zero
    const float c = g > 16.0f ? 16.0f : g < -16.0f ? -16.0f : g;
    return make_float2(g * s, fmaf(c * (s * (1.0f - s)), 1.5957691f * fmaf(0.134145f * c, c, 1.0f), s));
  }
}

// ---------------------------------------------------------------------------
// the kernel's arguments and units of work
// ---------------------------------------------------------------------------
struct GemmArgs {
  CUtensorMap a[2];          // forward: x; gradients: dgate, dup
  CUtensorMap b[3];          // Wg, Wu, x (gradients)
  int64_t rows, width, inner;
  // forward: `tiles` x `splits` units.  Gradients: units of dx (first), then of dWg and dWu
  int32_t tiles_m, tiles_n, splits;            // forward, or dx
  int32_t tiles_wm, tiles_wn, splits_w;        // dW: tile rows of one weight, tile columns, splits
  int32_t units, units_w;                      // of the first kind, of dW
  int32_t rounds_w, few_w;                     // dW units: rounds over all pairs, then those for pairs with one dx unit less
  // forward
  void *h, *gate, *up;
  uint8_t *gate_scale, *up_scale;
  int64_t ld_h, ld_gate, ld_up;
  const void* dh;            // backward
  int64_t ld_dh;
  const uint32_t* dh_max;    // fp16: dh_max_kernel's `dh_parts` maxima
  int32_t dh_parts;
  void *dgate, *dup;
  int64_t ld_d;
  // gradients
  void *dx, *dw[2];
  int64_t ld_dx, ld_dw[2];
  float* part;               // partial sums of the forward or of dx, or null; ld_part apart
  float* part_w;             // of dW
  int64_t ld_part;
  int32_t vec_h, vec_gate, vec_up, vec_dh, vec_dx, vec_dw[2];
  int32_t act, saved, dw_f32, accumulate;
  WsHeader* hdr;
};

using Yes = std::true_type;
using No = std::false_type;

struct Unit {
  int32_t kind;          // 0: the forward or dx, 1: dWg, 2: dWu
  int32_t m0, n0;        // tile's first row and column
  int32_t kb0, kb1;      // K blocks
  int32_t split;
};

template <int GROUP>
__device__ __forceinline__ void raster(int tile, int tiles_m, int tiles_n, int* tm, int* tn) {
  const int per = GROUP * tiles_n, g = tile / per, r = tile - g * per;
  const int gm = tiles_m - g * GROUP < GROUP ? tiles_m - g * GROUP : GROUP;
  *tn = r / gm;
  *tm = g * GROUP + (r - *tn * gm);
}

__device__ __forceinline__ int blocks_of(int64_t k) { return (int)((k + kBK - 1) / kBK); }

// The i-th unit of CTA pair `pair` out of `pairs`; false behind its last one.
template <int KIND, int NI>
__device__ __forceinline__ bool unit_at(const GemmArgs& A, int pair, int pairs, int i, Unit* u) {
  const int64_t first = (int64_t)i * pairs + pair;
  int tm, tn;
  if (KIND != K_GRAD || first < A.units) {
    if (first >= A.units) return false;
    const int tile = (int)first / A.splits;
    u->split = (int)first - tile * A.splits;
    raster<group_rows(KIND)>(tile, A.tiles_m, A.tiles_n, &tm, &tn);
    u->kind = 0;
    u->m0 = tm * kTile;
    u->n0 = tn * (KIND == K_GRAD ? kTile : NI);
    const int kb = KIND == K_GRAD ? 2 * blocks_of(A.inner) : blocks_of(A.width);
    u->kb0 = (int)((int64_t)kb * u->split / A.splits);
    u->kb1 = (int)((int64_t)kb * (u->split + 1) / A.splits);
    return true;
  }
  if (KIND == K_GRAD) {
    // dW units: whole rounds, then the share of the pairs that have one unit of dx less, then one more at most
    const int extra = A.units % pairs;                       // pairs [0, extra) have one unit of dx more
    const int done = A.units / pairs + (pair < extra ? 1 : 0);
    int j = i - done;
    int64_t w;
    if (j < A.rounds_w) {
      w = (int64_t)j * pairs + pair;
    } else {
      j -= A.rounds_w;
      const int few = pairs - extra;
      const int64_t base = (int64_t)A.rounds_w * pairs;
      if (pair >= extra && j < A.few_w) {
        w = base + (int64_t)j * few + (pair - extra);
      } else {
        if (pair >= extra) j -= A.few_w;
        w = base + (int64_t)A.few_w * few + (int64_t)j * pairs + pair;
      }
    }
    if (w >= A.units_w) return false;
    const int tile = (int)w / A.splits_w;
    u->split = (int)w - tile * A.splits_w;
    raster<group_rows(KIND)>(tile, 2 * A.tiles_wm, A.tiles_wn, &tm, &tn);
    const int second = tm >= A.tiles_wm;
    u->kind = 1 + second;
    u->m0 = (tm - (second ? A.tiles_wm : 0)) * kTile;
    u->n0 = tn * kTile;
    const int kb = blocks_of(A.rows);
    u->kb0 = (int)((int64_t)kb * u->split / A.splits_w);
    u->kb1 = (int)((int64_t)kb * (u->split + 1) / A.splits_w);
    return true;
  }
  return false;
}

// kind::f16: fp32 accumulator, A and B bf16 or fp16, M = 256, N columns.
template <int DT, int N>
__device__ __forceinline__ uint32_t instr_desc(bool a_mn, bool b_mn) {
  constexpr uint32_t type = DT == QMUON_BF16 ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}

// A thread's columns of gate and up: what the forward pass stores.  Every lane of the warp calls this.
template <int DT, int ACT, int W, bool ANY>
__device__ __forceinline__ void finish_forward(const GemmArgs& A, int64_t r, const Columns<W, ANY>& t, const float (&g)[W],
                                               const float (&u)[W]) {
  auto at = [&](void* base, int64_t ld) { return static_cast<unsigned char*>(base) + r * ld * elem_size(DT); };
  float h[W];
#pragma unroll
  for (int i = 0; i < W; ++i) h[i] = act_of<ACT>(g[i]) * u[i];
  t.template store<DT>(at(A.h, A.ld_h), A.vec_h, h);
  if (A.saved == QMUON_SAVE_SAME) {
    t.template store<DT>(at(A.gate, A.ld_gate), A.vec_gate, g);
    t.template store<DT>(at(A.up, A.ld_up), A.vec_up, u);
  } else if (A.saved == QMUON_SAVE_MXFP8) {
    const int64_t e = r * A.inner;
    encode_columns(t, static_cast<uint8_t*>(A.gate) + e, A.gate_scale + (e >> 5), A.vec_gate, g);
    encode_columns(t, static_cast<uint8_t*>(A.up) + e, A.up_scale + (e >> 5), A.vec_up, u);
  }
}
// The power of two that dgate and dup are held times: 1 but in fp16, where dh's largest finite magnitude is brought to
// [1/4, 1/2) if it lies below.  What is 2^-12 of it keeps all of its bits, and a smaller value is off by 2^-23 of it at most
// (times up act' or act); 1.3e5 times it still fits.  Never below 1: nothing is held with fewer bits than without.  Every
// lane of the warp calls this.
struct DhScale {
  float times, back;   // and its inverse
};
template <int DT>
__device__ __forceinline__ DhScale dh_scale(const GemmArgs& A) {
  if constexpr (DT != QMUON_FP16) return {1.0f, 1.0f};
  uint32_t m = 0;   // of fp32, not negative: ordered as integers
  for (int i = threadIdx.x & 31; i < A.dh_parts; i += 32) m = max(m, A.dh_max[i]);
  const uint32_t e = __reduce_max_sync(0xffffffffu, m) >> 23;   // 103 at least, or 0 for zero
  if (e == 0 || e >= 125) return {1.0f, 1.0f};
  return {__uint_as_float((252 - e) << 23), __uint_as_float((e + 2) << 23)};
}
// The same of the backward pass, from dh's words: dgate and dup for the products, and h again.
template <int DT, int ACT, int W, bool ANY>
__device__ __forceinline__ void finish_backward(const GemmArgs& A, int64_t r, const Columns<W, ANY>& t, const float (&g)[W],
                                                const float (&u)[W], const uint32_t (&dh)[W / 2], DhScale scale) {
  float h[W], dg[W], du[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float2 a = act_and_slope<ACT>(g[i]), d = unpack2<DT>(dh[i >> 1]);
    const float x = (i & 1 ? d.y : d.x) * scale.times;   // exact
    h[i] = a.x * u[i];
    dg[i] = x * u[i] * a.y;
    du[i] = x * a.x;
  }
  const int64_t e = r * A.ld_d * elem_size(DT);   // the workspace's rows are padded to 32 bytes
  t.template store<DT>(static_cast<unsigned char*>(A.dgate) + e, 2, dg);
  t.template store<DT>(static_cast<unsigned char*>(A.dup) + e, 2, du);
  if (A.h) t.template store<DT>(static_cast<unsigned char*>(A.h) + r * A.ld_h * elem_size(DT), A.vec_h, h);
}
// A thread's columns of dh as words.
template <int DT, int W, bool ANY>
__device__ __forceinline__ void load_dh(const GemmArgs& A, int64_t r, const Columns<W, ANY>& t, uint32_t (&w)[W / 2]) {
  const unsigned char* row = static_cast<const unsigned char*>(A.dh) + r * A.ld_dh * elem_size(DT);
  if (!ANY && A.vec_dh && t.n == W) {
    const uint4* p = reinterpret_cast<const uint4*>(row + t.c * elem_size(DT));
#pragma unroll
    for (int i = 0; i < W / 8; ++i) {
      const uint4 q = p[i];
      w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
    }
  } else {
    float v[W];
    t.template load<DT>(row, A.vec_dh, v);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) w[i] = pack2<DT>(v[2 * i], v[2 * i + 1]);
  }
}

// The q-th N elements of an array.
template <int N, class T, int M>
__device__ __forceinline__ const T (&part_of(const T (&v)[M], int q))[N] {
  return *reinterpret_cast<const T(*)[N]>(v + N * q);
}

// A wait of a whole warp, whose lanes go on together or not at all: tried in line, then bounded.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, WsHeader* h, unsigned where) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, h, where));
}

// NI: columns of gate, and of up, in a forward tile, 128 or 64 (see pick_tiles).
template <int KIND, int DT, int ACT, int NI>
__global__ void __launch_bounds__(kThreads, 1) ffn_kernel(const __grid_constant__ GemmArgs A) {
  constexpr int N = KIND == K_GRAD ? kTile : 2 * NI;             // columns of an accumulator
  constexpr int kBoxesB = N / 128;                               // of 64 of them, per CTA and stage
  constexpr uint32_t kLoadBytes = 2 * (2 + kBoxesB) * kBox;      // of both CTAs per stage
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 4);
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + kStages);
  const uint32_t tfull0 = smem_u32(bars + 2 * kStages), tempty0 = smem_u32(bars + 2 * kStages + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 2 * kEpiWarps);   // one arrival per epilogue warp of the pair
    }
    fence_mbar_init();
  }
  // the tensor maps that this call reads, ahead of the first copies
  if (KIND != K_GRAD) {
    if (warp == 0 && lane < 2) prefetch_map(lane == 0 ? &A.a[0] : &A.b[rank]);
  } else if (warp == 0 && lane < 5) {
    if (lane < 2) prefetch_map(&A.a[lane]);
    else if (lane < 4 ? A.units > 0 : A.units_w > 0) prefetch_map(&A.b[lane - 2]);
  }
  if (warp == 1) {
    tmem_alloc_cg<2>(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_cg<2>();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();   // the peer's barriers exist before anyone signals them
  tc_fence_after();
  depends_begin();
  const uint32_t tmem = *tmem_slot;
  const int inner_blocks = KIND == K_GRAD ? blocks_of(A.inner) : 0;

  // Warps 0 and 1 run a K block of 64 in the tensor cores' 512 cycles or hold
  // them up.  All lanes go through their loops, so that addresses, descriptors
  // and parities stay in uniform registers, where the TMA and MMA instructions
  // want them; one lane issues.  Stages are counted, not divided out, and a
  // barrier is tried in line before the bounded wait is called.
  if (warp == 0) {
    // ---- TMA producer: every CTA loads its own halves of the operands ----
    const uint32_t full_l = cluster_map(full0, 0);   // the leader's barriers
    const uint32_t smem0 = smem_u32(smem);
    int s = 0, it = 0;
    uint32_t parity = 1;   // of the round before: a new barrier's wait on it returns at once
    Unit u;
    // one unit's loads: A at (x, y) + (64 of its rows or columns), likewise B
    auto load = [&](auto a_mn, auto b_mn, const CUtensorMap* ma, const CUtensorMap* mb, int am, int bn, int k0, int n) -> bool {
      for (; n > 0; --n, ++it, k0 += kBK) {
        const uint32_t empty = empty0 + 8 * s, bar = full_l + 8 * s;
        if (!warp_wait(empty, parity, A.hdr, 0x2100u | KIND)) return false;
        const uint32_t sa = smem0 + s * kStageBytes;
        if (elect_one()) {
          if (leader) mbar_expect_tx(full0 + 8 * s, kLoadBytes);
          if constexpr (decltype(a_mn)::value) {
            tma_load_2d_pair(sa, ma, bar, am, k0);
            tma_load_2d_pair(sa + kBox, ma, bar, am + 64, k0);
          } else {
            tma_load_2d_pair(sa, ma, bar, k0, am);
            tma_load_2d_pair(sa + kBox, ma, bar, k0, am + 64);
          }
          if constexpr (decltype(b_mn)::value) {
            tma_load_2d_pair(sa + 2 * kBox, mb, bar, bn, k0);
            tma_load_2d_pair(sa + 3 * kBox, mb, bar, bn + 64, k0);
          } else {
            tma_load_2d_pair(sa + 2 * kBox, mb, bar, k0, bn);
            if constexpr (kBoxesB > 1) tma_load_2d_pair(sa + 3 * kBox, mb, bar, k0, bn + 64);
          }
        }
        __syncwarp();
        if (++s == kStages) s = 0, parity ^= 1;
      }
      return true;
    };
    for (int i = 0; unit_at<KIND, NI>(A, pair, pairs, i, &u); ++i) {
      const int am = u.m0 + 128 * rank;
      bool ok;
      if constexpr (KIND != K_GRAD) {
        ok = load(No{}, No{}, &A.a[0], &A.b[rank], am, u.n0, u.kb0 * kBK, u.kb1 - u.kb0);
      } else if (u.kind > 0) {
        ok = load(Yes{}, Yes{}, &A.a[u.kind - 1], &A.b[2], am, u.n0 + 128 * rank, u.kb0 * kBK, u.kb1 - u.kb0);
      } else {
        // dx runs over the columns of dgate, then over those of dup
        const int turn = inner_blocks < u.kb0 ? u.kb0 : inner_blocks > u.kb1 ? u.kb1 : inner_blocks;
        ok = load(No{}, Yes{}, &A.a[0], &A.b[0], am, u.n0 + 128 * rank, u.kb0 * kBK, turn - u.kb0) &&
             load(No{}, Yes{}, &A.a[1], &A.b[1], am, u.n0 + 128 * rank, (turn - inner_blocks) * kBK, u.kb1 - turn);
      }
      if (!ok) break;
    }
    // every load issued has landed before the CTA may exit (the leader's
    // full barriers also count the peer's loads)
    if (leader)
      for (int k = it > kStages ? it - kStages : 0; k < it; ++k)
        mbar_wait(full0 + 8 * (k % kStages), (k / kStages) & 1, A.hdr, 0x2200u | KIND);
  } else if (warp == 1) {
    if (leader) {
      // ---- MMA issuer ----
      // descriptors of the first stage: the low words hold the address, to which
      // 2 KB (MN-major) or 32 bytes (K-major) per 16 of K and a stage's 32 KB are added
      const uint32_t smem0 = smem_u32(smem);
      int s = 0;
      uint32_t parity = 0;
      auto multiply = [&](auto a_mn, auto b_mn, uint32_t d, int n) -> bool {
        constexpr bool amn = decltype(a_mn)::value, bmn = decltype(b_mn)::value;
        constexpr uint32_t step_a = (amn ? 2048 : 32) >> 4, step_b = (bmn ? 2048 : 32) >> 4;
        const uint64_t first_a = amn ? desc_mnmajor(smem0, 0) : desc_kmajor(smem0, 0);
        const uint64_t first_b = bmn ? desc_mnmajor(smem0 + 2 * kBox, 0) : desc_kmajor(smem0 + 2 * kBox, 0);
        const uint32_t idesc = instr_desc<DT, N>(amn, bmn);
        for (uint32_t add = 0; n > 0; --n, add = 1) {
          const uint32_t full = full0 + 8 * s;
          if (!warp_wait(full, parity, A.hdr, 0x2300u | KIND)) return false;
          tc_fence_after();
          const uint64_t ad = first_a + (uint32_t)(s * (kStageBytes >> 4)), bd = first_b + (uint32_t)(s * (kStageBytes >> 4));
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk) mma_bf16_cg<2>(d, ad + kk * step_a, bd + kk * step_b, idesc, kk > 0 ? 1u : add);
            mma_commit_cg<2>(empty0 + 8 * s);
          }
          __syncwarp();
          if (++s == kStages) s = 0, parity ^= 1;
        }
        return true;
      };
      Unit u;
      for (int i = 0; unit_at<KIND, NI>(A, pair, pairs, i, &u); ++i) {
        const int acc = i & 1, use = i >> 1;
        if (use > 0 && !warp_wait(tempty0 + 8 * acc, (use - 1) & 1, A.hdr, 0x2500u | KIND)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * kTile);
        bool ok;
        if constexpr (KIND != K_GRAD) ok = multiply(No{}, No{}, d, u.kb1 - u.kb0);
        else if (u.kind > 0) ok = multiply(Yes{}, Yes{}, d, u.kb1 - u.kb0);
        else ok = multiply(No{}, Yes{}, d, u.kb1 - u.kb0);
        if (elect_one()) mma_commit_cg<2>(tfull0 + 8 * acc);   // accumulator ready (also on the error path)
        __syncwarp();
        if (!ok) break;
      }
    }
  } else {
    // ---- epilogue: warps 2..9; TMEM lane quarter = warp % 4 ----
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tempty_l = cluster_map(tempty0, 0);
    DhScale scale{1.0f, 1.0f};
    if constexpr (KIND != K_FWD) scale = dh_scale<DT>(A);
    Unit u;
    for (int i = 0; unit_at<KIND, NI>(A, pair, pairs, i, &u); ++i) {
      const int64_t r = u.m0 + 128 * rank + quarter * 32 + lane;
      const int acc = i & 1, use = i >> 1;
      const int64_t c0 = u.n0 + (KIND != K_GRAD ? NI / 2 : 128) * half;   // this warp's first column
      uint32_t dh[KIND == K_BWD ? NI / 64 : 1][16];
      if (KIND == K_BWD && !A.part) {   // while the tensor cores work
#pragma unroll
        for (int j = 0; j < NI / 64; ++j) {
          const int64_t c = c0 + 32 * j;
          load_dh<DT, 32, false>(A, r, {c, r < A.rows ? valid_columns(A.inner - c, 32) : 0}, dh[j]);
        }
      }
      bool ok = mbar_wait(tfull0 + 8 * acc, use & 1, A.hdr, 0x2400u | KIND);
      tc_fence_after();
      ok = ok && *reinterpret_cast<volatile unsigned*>(&A.hdr->error) == 0u;
      if (!__all_sync(0xffffffffu, ok)) break;   // tcgen05.ld is warp-collective
      const uint32_t t = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * kTile);
      auto release = [&] {   // every TMEM read of this accumulator by this warp is done
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty_l + 8 * acc);
      };
      if (KIND != K_GRAD) {
#pragma unroll
        for (int j = 0; j < NI / 64; ++j) {
          uint32_t gv[32], uv[32];
          __syncwarp();   // lanes without a row rejoin: tcgen05.ld is warp-collective
          tmem_ld32_async(t + (uint32_t)(NI / 2 * half + 32 * j), gv);
          tmem_ld32_async(t + (uint32_t)(NI + NI / 2 * half + 32 * j), uv);
          tmem_wait_ld();
          tmem_hold(gv);
          tmem_hold(uv);
          if (j == NI / 64 - 1) release();
          float g[32], v[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) g[k] = __uint_as_float(gv[k]), v[k] = __uint_as_float(uv[k]);
          const int64_t c = c0 + 32 * j;
          const int n = r < A.rows ? valid_columns(A.inner - c, 32) : 0;
          if (A.part) {   // [split][gate, up][rows][ld_part]
            const int np = n ? valid_columns(A.ld_part - c, 32) : 0;
            float* p = A.part + (n ? (((int64_t)u.split * 2) * A.rows + r) * A.ld_part + c : 0);
            store_row<QMUON_FP32, 32>(p, np, 2, g);
            store_row<QMUON_FP32, 32>(p + A.rows * A.ld_part, np, 2, v);
          } else if constexpr (KIND == K_FWD) {
            finish_forward<DT, ACT, 32, false>(A, r, {c, n}, g, v);
          } else if constexpr (KIND == K_BWD) {
            // in halves: the registers do not hold 32 columns of everything
#pragma unroll
            for (int q = 0; q < 2; ++q)
              finish_backward<DT, ACT, 16, false>(A, r, {c + 16 * q, valid_columns(n - 16 * q, 16)}, part_of<16>(g, q),
                                                  part_of<16>(v, q), part_of<8>(dh[j], q), scale);
          }
        }
      } else {
        const int64_t rows = u.kind == 0 ? A.rows : A.inner;
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          uint32_t av[32];
          __syncwarp();
          tmem_ld32(t + (uint32_t)(128 * half + 32 * j), av);
          if (j == 3) release();
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(av[k]) * scale.back;
          const int64_t c = c0 + 32 * j;
          const int n = r < rows ? valid_columns(A.width - c, 32) : 0;
          float* part = u.kind == 0 ? A.part : A.part_w;
          if (part) {   // dx: [split][rows][ld_part]; dW: [weight][split][inner][ld_part]
            const int64_t slice = u.kind == 0 ? u.split : (int64_t)(u.kind - 1) * A.splits_w + u.split;
            store_row<QMUON_FP32, 32>(part + (n ? (slice * rows + r) * A.ld_part + c : 0), n ? valid_columns(A.ld_part - c, 32) : 0, 2, v);
          } else if (u.kind == 0) {
            store_row<DT, 32>(static_cast<unsigned char*>(A.dx) + (n ? (r * A.ld_dx + c) * elem_size(DT) : 0), n, A.vec_dx, v);
          } else {
            const int w = u.kind - 1;
            unsigned char* p = static_cast<unsigned char*>(A.dw[w]) + (n ? (r * A.ld_dw[w] + c) * (A.dw_f32 ? 4 : elem_size(DT)) : 0);
            if (A.accumulate) {
              float old[32];
              if (A.dw_f32) load_row<QMUON_FP32, 32>(p, n, A.vec_dw[w], old);
              else load_row<DT, 32>(p, n, A.vec_dw[w], old);
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] += old[k];
            }
            if (A.dw_f32) store_row<QMUON_FP32, 32>(p, n, A.vec_dw[w], v);
            else store_row<DT, 32>(p, n, A.vec_dw[w], v);
          }
        }
      }
    }
  }

  // ---- teardown: every accumulator read is done and the peer no longer
  // touches this CTA's barriers or shared memory ----
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<2>(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// element by element: gate and up from partial sums, from their 16-bit copies
// or from their carriers
// ---------------------------------------------------------------------------
constexpr int kElemThreads = 256, kElemCols = 16;
enum { FROM_PART = 0, FROM_SAME = 1, FROM_MXFP8 = 2 };

struct ElemArgs {
  GemmArgs A;            // outputs, dh, sizes
  const float* part;     // [splits][gate, up][rows][ld_part]
  int32_t splits;
  const void *gate, *up; // FROM_SAME and FROM_MXFP8
  const uint8_t *gate_scale, *up_scale;
  int64_t ld_gate, ld_up;
  int32_t vec_in;        // rows of gate and up
  int32_t clear;         // the workspace's header has not been cleared
};

// The workspace's header, by the first CTA of a kernel that is complete before any kernel looks at it.
__device__ __forceinline__ void clear_header(WsHeader* h) {
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < kWsHeader / 4) reinterpret_cast<uint32_t*>(h)[threadIdx.x] = 0u;
}

// The same as a kernel of its own, for calls that begin with the tensor-core kernel: unlike a memset's, its dependents'
// start overlaps it.
__global__ void __launch_bounds__(64) clear_kernel(WsHeader* h) {
  depends_begin();
  clear_header(h);
}
cudaError_t launch_clear(WsHeader* h, cudaStream_t s) { return launch_dependent(clear_kernel, dim3(1), dim3(64), 0, s, h); }

// A thread takes 16 columns of a row.  (Of 32, as in the product's epilogue, the 160 registers left 12 warps on an SM:
// 8192 x 14336 from carriers in 214 us.)
template <int DT, int ACT, int FROM, bool BWD, bool ANY>
__global__ void __launch_bounds__(kElemThreads) elem_kernel(const __grid_constant__ ElemArgs E) {
  constexpr int W = kElemCols, es = elem_size(DT);
  const GemmArgs& A = E.A;
  depends_begin();
  if (E.clear) clear_header(A.hdr);
  int64_t r;
  const Columns<W, ANY> t = deal_columns<W, ANY>((int64_t)blockIdx.x * kElemThreads + threadIdx.x, A.rows, A.inner, &r);
  uint32_t dh[W / 2];
  if constexpr (BWD) load_dh<DT, W, ANY>(A, r, t, dh);
  float g[W], u[W];
  if constexpr (FROM == FROM_PART) {
    const float* p = E.part + r * A.ld_part;
    t.template load<QMUON_FP32>(p, 2, g);
    t.template load<QMUON_FP32>(p + A.rows * A.ld_part, 2, u);
    for (int s = 1; s < E.splits; ++s) {
      p += 2 * A.rows * A.ld_part;
      float a[W], b[W];
      t.template load<QMUON_FP32>(p, 2, a);
      t.template load<QMUON_FP32>(p + A.rows * A.ld_part, 2, b);
#pragma unroll
      for (int k = 0; k < W; ++k) g[k] += a[k], u[k] += b[k];
    }
  } else if constexpr (FROM == FROM_SAME) {
    t.template load<DT>(static_cast<const unsigned char*>(E.gate) + r * E.ld_gate * es, E.vec_in, g);
    t.template load<DT>(static_cast<const unsigned char*>(E.up) + r * E.ld_up * es, E.vec_in, u);
  } else {
    const int64_t e = r * A.inner;
    decode_columns(t, static_cast<const uint8_t*>(E.gate) + e, E.gate_scale + (e >> 5), E.vec_in, g);
    decode_columns(t, static_cast<const uint8_t*>(E.up) + e, E.up_scale + (e >> 5), E.vec_in, u);
  }
  if constexpr (BWD) finish_backward<DT, ACT, W, ANY>(A, r, t, g, u, dh, dh_scale<DT>(A));
  else finish_forward<DT, ACT, W, ANY>(A, r, t, g, u);
}

// The largest finite magnitude of dh (fp16), one maximum per CTA as the bits of an fp32: a pass over dh of its own, before
// anything can be rounded.  Bound by DRAM: 50 us of 8192 x 14336 (4.7 TB/s; the call takes 2500), 3 of 2048 x 1024 (18 -> 21).
constexpr int kMaxThreads = 1024, kMaxCols = 16, kMaxUnroll = 2;
struct MaxArgs {
  const void* dh;
  int64_t rows, inner, ld, threads;
  int32_t vec;
  uint32_t* out;
};
template <bool ANY>
__global__ void __launch_bounds__(kMaxThreads) dh_max_kernel(MaxArgs A) {
  constexpr int W = kMaxCols;
  __shared__ uint32_t warp_max[kMaxThreads / 32];
  depends_begin();
  uint32_t m = 0;
  const int64_t step = (int64_t)gridDim.x * kMaxThreads;
  for (int64_t i = (int64_t)blockIdx.x * kMaxThreads + threadIdx.x; i < A.threads; i += kMaxUnroll * step) {
    float v[kMaxUnroll][W];
#pragma unroll
    for (int k = 0; k < kMaxUnroll; ++k) {
      int64_t r;
      const Columns<W, ANY> t = deal_columns<W, ANY>(i + k * step, A.rows, A.inner, &r);
      t.template load<QMUON_FP16>(static_cast<const unsigned char*>(A.dh) + r * A.ld * 2, A.vec, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kMaxUnroll; ++k)
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (fabsf(v[k][j]) <= 65504.0f) m = max(m, __float_as_uint(fabsf(v[k][j])));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x < 32) {
    m = __reduce_max_sync(0xffffffffu, warp_max[threadIdx.x]);
    if (threadIdx.x == 0) A.out[blockIdx.x] = m;
  }
}
static_assert(kMaxThreads == 32 * 32, "a warp reduces the warps' maxima");

// Sums of split products, rows x cols of [splits][rows][ld_part], to the type of the result; the products of a call
// together in one launch.
constexpr int kJoinCols = 8;
struct Join {
  const float* part;
  void* out;
  int64_t rows, cols, ld_part, ld, first;   // first: its first CTA
  int32_t splits, vec, accumulate, dt;
};
struct JoinArgs {
  Join job[3];
  int32_t n;
};
template <int DT, bool ANY>
__device__ __forceinline__ void join_columns(const Join& J, int64_t i) {
  constexpr int W = kJoinCols;
  int64_t r;
  const Columns<W, ANY> t = deal_columns<W, ANY>(i, J.rows, J.cols, &r);
  const float* p = J.part + r * J.ld_part;
  float v[W];
  t.template load<QMUON_FP32>(p, 2, v);
#pragma unroll 4
  for (int s = 1; s < J.splits; ++s) {
    float a[W];
    t.template load<QMUON_FP32>(p + s * J.rows * J.ld_part, 2, a);
#pragma unroll
    for (int k = 0; k < W; ++k) v[k] += a[k];
  }
  unsigned char* o = static_cast<unsigned char*>(J.out) + r * J.ld * elem_size(DT);
  if (J.accumulate) {
    float old[W];
    t.template load<DT>(o, J.vec, old);
#pragma unroll
    for (int k = 0; k < W; ++k) v[k] += old[k];
  }
  t.template store<DT>(o, J.vec, v);
}
template <int DT>
__device__ __forceinline__ void join_one(const Join& J, int64_t i) {
  if (J.vec) join_columns<DT, false>(J, i);
  else join_columns<DT, true>(J, i);
}
__global__ void __launch_bounds__(kElemThreads) join_kernel(const __grid_constant__ JoinArgs A) {
  depends_begin();
  const Join& J = A.job[A.n > 2 && blockIdx.x >= A.job[2].first ? 2 : A.n > 1 && blockIdx.x >= A.job[1].first ? 1 : 0];
  const int64_t i = ((int64_t)blockIdx.x - J.first) * kElemThreads + threadIdx.x;
  if (J.dt == QMUON_BF16) join_one<QMUON_BF16>(J, i);
  else if (J.dt == QMUON_FP16) join_one<QMUON_FP16>(J, i);
  else join_one<QMUON_FP32>(J, i);
}

// ---------------------------------------------------------------------------
// few rows: the weights once through the cores' registers
// ---------------------------------------------------------------------------
// With few rows the time is the weights' way from DRAM.  A CTA takes 8 columns
// of gate and the same 8 of up, as the 16 rows of an m16n8k16 product whose 8
// columns are rows of x (NT such products for 8 NT rows; more rows are other
// CTAs', grid.y): gate and up of a
// column meet in one thread.  Its 8 warps take turns over K, 32 at a time: a
// lane loads 16 bytes of a row of Wg, of Wu and of x at the same columns, in
// which order K is summed does not matter, so the pieces go straight into the
// operands' registers.  The warps' sums are added through shared memory in
// order.  (The CTA pairs above leave it to a few SMs' loads in flight: one row of
// 4096 x 14336 took 70 us.)
constexpr int kFewThreads = 256, kFewCols = 8, kFewRows = 16;

struct FewArgs {
  GemmArgs A;
  const void *x, *w[2];
  int64_t ld_x, ld_w[2];
};

template <int DT>
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (DT == QMUON_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 elements from column k of a row of `width`, zeros behind its end and where the row is not there.  ONCE: not kept in L1.
template <bool VEC, bool ONCE>
__device__ __forceinline__ uint4 eight_of(const uint16_t* row, bool there, int64_t k, int64_t width) {
  uint4 q = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (VEC) {
    if (!there || k >= width) return q;
    if constexpr (ONCE)
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "l"(row + k) : "memory");
    else
      q = *reinterpret_cast<const uint4*>(row + k);
  } else {
    const int n = there ? valid_columns(width - k, 8) : 0;
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < n ? row[k + i] : 0u;
    q = make_uint4(e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16), e[6] | (e[7] << 16));
  }
  return q;
}

template <int DT, int ACT, int NT, bool VEC>
__global__ void __launch_bounds__(kFewThreads, 3) few_kernel(const __grid_constant__ FewArgs F) {
  const GemmArgs& A = F.A;
  constexpr int kWarps = kFewThreads / 32, U = 2;   // U steps of K at a time
  __shared__ float4 sums[kWarps][NT * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t j = (int64_t)blockIdx.x * kFewCols + g, row0 = (int64_t)blockIdx.y * (8 * NT);
  const bool there = j < A.inner;
  const uint16_t* wg = static_cast<const uint16_t*>(F.w[0]) + (there ? j : 0) * F.ld_w[0];
  const uint16_t* wu = static_cast<const uint16_t*>(F.w[1]) + (there ? j : 0) * F.ld_w[1];
  const int64_t steps = (A.width + 31) >> 5;
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
  depends_begin();
  clear_header(A.hdr);
  uint4 a[U], b[U];
  auto load = [&](int64_t s0, uint4 (&to_a)[U], uint4 (&to_b)[U]) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t k = (s0 + i * kWarps) * 32 + 8 * t;
      to_a[i] = eight_of<VEC, true>(wg, there, k, A.width);
      to_b[i] = eight_of<VEC, true>(wu, there, k, A.width);
    }
  };
  load(warp, a, b);
  for (int64_t s0 = warp; s0 < steps; s0 += kWarps * U) {
    uint4 next_a[U], next_b[U];   // on their way while these are multiplied
    load(s0 + kWarps * U, next_a, next_b);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t k = (s0 + i * kWarps) * 32 + 8 * t;
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        const int64_t row = row0 + 8 * m + g;
        const uint4 x = eight_of<VEC, false>(static_cast<const uint16_t*>(F.x) + (row < A.rows ? row : 0) * F.ld_x, row < A.rows, k, A.width);
        mma_16x8x16<DT>(acc[m], a[i].x, b[i].x, a[i].y, b[i].y, x.x, x.y);
        mma_16x8x16<DT>(acc[m], a[i].z, b[i].z, a[i].w, b[i].w, x.z, x.w);
      }
      a[i] = next_a[i], b[i] = next_b[i];
    }
  }
#pragma unroll
  for (int m = 0; m < NT; ++m) sums[warp][m * 32 + lane] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
  __syncthreads();
  if (threadIdx.x >= NT * 32 || !there) return;
  float4 v = sums[0][threadIdx.x];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) {
    const float4 q = sums[w][threadIdx.x];
    v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {   // gate and up of column j, rows 2 t and 2 t + 1 of this thread's product
    const int64_t row = row0 + 8 * warp + 2 * t + i;
    if (row >= A.rows) break;
    const float gate = i ? v.y : v.x, up = i ? v.w : v.z;
    if (A.part) {   // [gate, up][rows][ld_part]
      A.part[row * A.ld_part + j] = gate;
      A.part[(A.rows + row) * A.ld_part + j] = up;
    } else {
      store_elem<DT>(A.h, row * A.ld_h + j, act_of<ACT>(gate) * up);
      if (A.saved == QMUON_SAVE_SAME) {
        store_elem<DT>(A.gate, row * A.ld_gate + j, gate);
        store_elem<DT>(A.up, row * A.ld_up + j, up);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// rows x cols of 16-bit elements, boxes of 64 x 64, 128-byte swizzle.
bool encode_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int dt) {
  EncodeTiledFn fn = encoder();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, 64};
  cuuint32_t es[2] = {1, 1};
  const CUresult r =
      fn(m, dt == QMUON_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims,
         strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r == CUDA_SUCCESS) return true;
  char msg[256];
  std::snprintf(msg, sizeof(msg), "cuTensorMapEncodeTiled returned %d for a %lld x %lld matrix (row stride %lld) at %p", (int)r,
                (long long)rows, (long long)cols, (long long)ld, base);
  set_error_msg(msg, QMUON_ERR_CUDA);
  return false;
}

// A tensor map reads rows that start on 16 bytes; others are copied to the workspace first.
bool tma_ready(const void* p, int64_t ld) { return is_aligned(p, 16) && ld % 8 == 0; }

// The most K blocks of a unit, 5.4e8 cycles of the tensor cores: the epilogue waits for all of them at once, and its wait
// is bounded (kWaitCycles, 4e9).  dx over 2^28 columns of dgate and of dup, 2^23 blocks, would outlast it in one piece.
constexpr int kMaxBlocks = 1 << 20;
static_assert((long long)kMaxBlocks * 512 * 4 < kWaitCycles, "a unit ends long before its wait does");

// The width of the projections' tiles and the splits of their K blocks: the least estimated time, in twentieths of a K
// block of a pair on a tile of 128 columns.  A block of 64 columns takes 12 (its rows' operand is as large), a unit 20 more,
// the last epilogue 200 or 100, partial sums 40 a unit and 160 for their kernel.  Narrow tiles are for what fills the pairs
// badly, and for short K, where the last epilogue counts: 100 x 4096 x 512 13.2 us against 19.0, 2000 x 256 x 1024 8.1
// against 8.8, 4000 x 512 x 512 9.4 against 10.3, 64 x 4096 x 14336 46.6 against 48.4; wide ones for the rest: 300 x 1000 x
// 3000 16.2 against 18.4, 1024 x 4096 x 14336 123 against 149.
struct Tiles {
  int inner, splits;
};
Tiles pick_tiles(int64_t rows, int64_t width, int64_t inner, int pairs) {
  const int64_t kb = ceil_div(width, kBK);
  Tiles best{128, 1};
  int64_t best_cost = INT64_MAX;
  for (const int ni : {128, 64}) {
    const int64_t tiles = ceil_div(rows, kTile) * ceil_div(inner, ni), block = ni == 128 ? 20 : 12, last = ni == 128 ? 200 : 100;
    const int least = (int)ceil_div(kb, kMaxBlocks);
    const int most = tiles >= pairs ? least : (int)std::min<int64_t>(32, std::max<int64_t>(1, kb / 4));
    for (int s = least; s <= most; ++s) {
      const int64_t cost =
          ceil_div(tiles * s, pairs) * (ceil_div(kb, s) * block + 20 + (s > 1 ? 40 : 0)) + last + (s > 1 ? 160 : 0);
      if (cost < (ni == best.inner ? best_cost : best_cost * 9 / 10)) best_cost = cost, best = Tiles{ni, s};   // narrow: only where it is clear
    }
  }
  return best;
}

struct Geometry {
  int pairs = 0;
  int32_t tiles_m = 0, tiles_n = 0, splits = 1;         // forward (or the projections again)
  int32_t inner_tile = 128;
  int32_t dx_m = 0, dx_n = 0, dx_splits = 1;
  int32_t dw_m = 0, dw_n = 0, dw_splits = 1;
  int64_t ld_fwd = 0, ld_w = 0, ld_d = 0;               // of partial gate/up, of partial dx/dW, of dgate/dup
  size_t dgate = 0, dup = 0, dh_max = 0, x = 0, w[2] = {0, 0}, part = 0, part_x = 0, part_w = 0, total = 0;
  int64_t ld_x = 0, ld_wp = 0;
  bool copy_x = false, copy_w[2] = {false, false};
  bool few = false;                                     // the projections by few_kernel
};

// Whether few_kernel makes the projections.  Up to 16 rows: one pass over the weights (4096 x 14336 34 us, the CTA pairs
// 60; 32 rows in one pass 70).  More rows read the weights again for every 16, out of L2, which pays where the pairs' fixed
// 6 us (tensor memory, a cluster's start, the header's clearing) are the larger part: 64 x 256 x 1024 3.3 us against 6.6,
// 128 x 512 x 512 3.5 against 8.0, but 256 x 256 x 1024 7.7 against 7.1 and 64 x 256 x 8192 13.5 against 7.6; with rows
// off 16 bytes 64 x 256 x 1024 6.6 against 8.0, 128 x 256 x 1024 10.2 against 8.5.
bool few_rows(int64_t rows, int64_t width, int64_t inner, bool vec) {
  if (rows <= kFewRows) return true;
  const int64_t most = vec ? (int64_t)1 << 26 : (int64_t)3 << 23;
  return rows <= 4096 && inner <= most / rows / width;
}

// What a call lays out in its workspace, behind the header.
void lay(Geometry& G, size_t* at, size_t bytes) { *at = G.total, G.total += round_up(bytes, 256); }

void lay_operands(Geometry& G, int64_t rows, int64_t width, int64_t inner, bool x, bool wg, bool wu) {
  G.copy_x = x;
  G.copy_w[0] = wg;
  G.copy_w[1] = wu;
  G.ld_x = G.ld_wp = (int64_t)round_up((size_t)width, 8);
  if (x) lay(G, &G.x, (size_t)rows * G.ld_x * 2);
  for (int i = 0; i < 2; ++i)
    if (G.copy_w[i]) lay(G, &G.w[i], (size_t)inner * G.ld_wp * 2);
}

// `direct`: the product's own kernel may finish a column of gate and up; else their fp32 values go through the workspace
// to elem_kernel, as split products' do.  The tensor-core kernel's epilogue has 8 warps on an SM and accesses rows in
// vectors only (written by elements there, the rows of fp16 3001 x 2731 took 45 us); few_kernel writes by elements, but
// no codes.
void lay_projections(Geometry& G, int64_t rows, int64_t width, int64_t inner, bool direct) {
  G.ld_fwd = (int64_t)round_up((size_t)inner, 8);
  if (G.few) {
    if (!direct) lay(G, &G.part, (size_t)2 * rows * G.ld_fwd * 4);
    return;
  }
  G.tiles_m = (int32_t)ceil_div(rows, kTile);
  const Tiles t = pick_tiles(rows, width, inner, G.pairs);
  G.inner_tile = t.inner;
  G.tiles_n = (int32_t)ceil_div(inner, t.inner);
  G.splits = t.splits;
  if (G.splits > 1 || !direct) lay(G, &G.part, (size_t)G.splits * 2 * rows * G.ld_fwd * 4);
}

Geometry forward_geometry(const qmuon_gated_ffn& c, int pairs) {
  Geometry G;
  G.pairs = pairs;
  G.total = kWsHeader;
  G.few = few_rows(c.rows, c.width, c.inner, tma_ready(c.x, c.ld_x) && tma_ready(c.w_gate, c.ld_w_gate) && tma_ready(c.w_up, c.ld_w_up));
  if (!G.few)
    lay_operands(G, c.rows, c.width, c.inner, !tma_ready(c.x, c.ld_x), !tma_ready(c.w_gate, c.ld_w_gate), !tma_ready(c.w_up, c.ld_w_up));
  const bool vectors = vec_class(c.h, c.ld_h, 2) &&
                       (c.saved != QMUON_SAVE_SAME || (vec_class(c.gate, c.ld_gate, 2) && vec_class(c.up, c.ld_up, 2)));
  lay_projections(G, c.rows, c.width, c.inner, G.few ? c.saved != QMUON_SAVE_MXFP8 : vectors);
  return G;
}

// What the backward pass reads besides dh and what was saved.
bool needs_x(const qmuon_gated_ffn_grad& c) { return c.dw_gate || c.saved == QMUON_SAVE_NONE; }
bool needs_weights(const qmuon_gated_ffn_grad& c) { return c.dx || c.saved == QMUON_SAVE_NONE; }

Geometry backward_geometry(const qmuon_gated_ffn_grad& c, int pairs) {
  Geometry G;
  G.pairs = pairs;
  G.total = kWsHeader;
  G.few = few_rows(c.rows, c.width, c.inner,
                   (c.x_scale || tma_ready(c.x, c.ld_x)) && tma_ready(c.w_gate, c.ld_w_gate) && tma_ready(c.w_up, c.ld_w_up));
  const bool w = c.dx || (c.saved == QMUON_SAVE_NONE && !G.few);   // few_kernel reads them as they are
  lay_operands(G, c.rows, c.width, c.inner, needs_x(c) && (c.x_scale || ((c.dw_gate || !G.few) && !tma_ready(c.x, c.ld_x))),
               w && !tma_ready(c.w_gate, c.ld_w_gate), w && !tma_ready(c.w_up, c.ld_w_up));
  G.ld_d = (int64_t)round_up((size_t)c.inner, 16);
  lay(G, &G.dgate, (size_t)c.rows * G.ld_d * 2);
  lay(G, &G.dup, (size_t)c.rows * G.ld_d * 2);
  if (c.dtype == QMUON_FP16) lay(G, &G.dh_max, (size_t)2 * G.pairs * 4);
  G.ld_w = (int64_t)round_up((size_t)c.width, 8);
  const size_t behind = G.total;
  if (c.saved == QMUON_SAVE_NONE)
    lay_projections(G, c.rows, c.width, c.inner, !G.few && vec_class(c.dh, c.ld_dh, 2) && (!c.h || vec_class(c.h, c.ld_h, 2)));
  const size_t most = G.total;
  G.total = behind;   // the projections' partial sums are done with when the gradients' begin
  const int kbx = 2 * (int)ceil_div(c.inner, kBK), kbw = (int)ceil_div(c.rows, kBK);
  if (c.dx) {
    G.dx_m = (int32_t)ceil_div(c.rows, kTile);
    G.dx_n = (int32_t)ceil_div(c.width, kTile);
  }
  if (c.dw_gate) {
    G.dw_m = (int32_t)ceil_div(c.inner, kTile);
    G.dw_n = (int32_t)ceil_div(c.width, kTile);
  }
  const int64_t tx = (int64_t)G.dx_m * G.dx_n, tw = 2 * (int64_t)G.dw_m * G.dw_n;
  if (tx + tw < 2 * (int64_t)G.pairs) {
    // few tiles: units of at most `most` K blocks, of whole tiles or of a pair's share of all blocks and its multiples,
    // whichever is estimated to end first (the longest unit, or all of them over the pairs; partial sums cost about 16
    // blocks for their way through memory and their kernel)
    const int64_t all = tx * kbx + tw * kbw, share = std::max<int64_t>(4, ceil_div(all, G.pairs));
    int64_t best = INT64_MAX;
    for (const int64_t most : {(int64_t)1 << 40, 4 * share, 2 * share, share}) {
      const int64_t sx = tx ? std::min<int64_t>(32, ceil_div(kbx, most)) : 1, sw = tw ? std::min<int64_t>(32, ceil_div(kbw, most)) : 1;
      const int64_t longest = std::max(tx ? ceil_div(kbx, sx) : 0, tw ? ceil_div(kbw, sw) : 0) + 6, units = tx * sx + tw * sw;
      const int64_t cost = std::max(longest, ceil_div(units, G.pairs) * (ceil_div(all, units) + 6)) + (sx > 1 || sw > 1 ? 16 : 0);
      if (cost < best) best = cost, G.dx_splits = (int32_t)sx, G.dw_splits = (int32_t)sw;
    }
  }
  G.dx_splits = std::max(G.dx_splits, (int32_t)ceil_div(kbx, kMaxBlocks));
  G.dw_splits = std::max(G.dw_splits, (int32_t)ceil_div(kbw, kMaxBlocks));
  const int gs = elem_size(c.grad_dtype);
  if (c.dx && (G.dx_splits > 1 || !vec_class(c.dx, c.ld_dx, 2))) lay(G, &G.part_x, (size_t)G.dx_splits * c.rows * G.ld_w * 4);
  if (c.dw_gate && (G.dw_splits > 1 || !vec_class(c.dw_gate, c.ld_dw_gate, gs) || !vec_class(c.dw_up, c.ld_dw_up, gs)))
    lay(G, &G.part_w, (size_t)2 * G.dw_splits * c.inner * G.ld_w * 4);
  G.total = std::max(G.total, most);
  return G;
}

template <class K>
cudaError_t launch_pairs(K kernel, const GemmArgs& A, int64_t units, int pairs, cudaStream_t s) {
  // the shared-memory limit is per device; setting it again costs a few hundred nanoseconds
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(units, pairs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, A);
}

template <int KIND, int DT, int NI>
cudaError_t launch_act(const GemmArgs& A, int64_t units, int pairs, cudaStream_t s) {
  if (A.act == QMUON_ACT_SILU) return launch_pairs(ffn_kernel<KIND, DT, QMUON_ACT_SILU, NI>, A, units, pairs, s);
  if (A.act == QMUON_ACT_GELU) return launch_pairs(ffn_kernel<KIND, DT, QMUON_ACT_GELU, NI>, A, units, pairs, s);
  return launch_pairs(ffn_kernel<KIND, DT, QMUON_ACT_GELU_TANH, NI>, A, units, pairs, s);
}
template <int KIND>
cudaError_t launch_projections(const GemmArgs& A, const Geometry& G, int dt, cudaStream_t s) {
  if (G.inner_tile == 128)
    return dt == QMUON_BF16 ? launch_act<KIND, QMUON_BF16, 128>(A, A.units, G.pairs, s) : launch_act<KIND, QMUON_FP16, 128>(A, A.units, G.pairs, s);
  return dt == QMUON_BF16 ? launch_act<KIND, QMUON_BF16, 64>(A, A.units, G.pairs, s) : launch_act<KIND, QMUON_FP16, 64>(A, A.units, G.pairs, s);
}
cudaError_t launch_gradients(const GemmArgs& A, int64_t units, int pairs, int dt, cudaStream_t s) {
  return dt == QMUON_BF16 ? launch_pairs(ffn_kernel<K_GRAD, QMUON_BF16, 0, 128>, A, units, pairs, s)
                          : launch_pairs(ffn_kernel<K_GRAD, QMUON_FP16, 0, 128>, A, units, pairs, s);
}

template <int DT, int FROM, bool BWD>
cudaError_t launch_elem_of(const ElemArgs& E, cudaStream_t s) {
  const bool vec = (!BWD || E.A.vec_dh) && (FROM != FROM_SAME || E.vec_in) && (!E.A.h || E.A.vec_h) &&
                   (BWD || E.A.saved != QMUON_SAVE_SAME || (E.A.vec_gate && E.A.vec_up));
  const int64_t grid = ceil_div(threads_of(E.A.rows, E.A.inner, kElemCols, !vec), kElemThreads);
  auto go = [&](auto kernel, auto any) { return launch_dependent(vec ? kernel : any, dim3((unsigned)grid), dim3(kElemThreads), 0, s, E); };
  if (E.A.act == QMUON_ACT_SILU) return go(elem_kernel<DT, QMUON_ACT_SILU, FROM, BWD, false>, elem_kernel<DT, QMUON_ACT_SILU, FROM, BWD, true>);
  if (E.A.act == QMUON_ACT_GELU) return go(elem_kernel<DT, QMUON_ACT_GELU, FROM, BWD, false>, elem_kernel<DT, QMUON_ACT_GELU, FROM, BWD, true>);
  return go(elem_kernel<DT, QMUON_ACT_GELU_TANH, FROM, BWD, false>, elem_kernel<DT, QMUON_ACT_GELU_TANH, FROM, BWD, true>);
}
template <int FROM, bool BWD>
cudaError_t launch_elem(const ElemArgs& E, int dt, cudaStream_t s) {
  return dt == QMUON_BF16 ? launch_elem_of<QMUON_BF16, FROM, BWD>(E, s) : launch_elem_of<QMUON_FP16, FROM, BWD>(E, s);
}

void add_join(JoinArgs& A, int64_t* grid, const float* part, int splits, int64_t rows, int64_t cols, int64_t ld_part, void* out, int64_t ld,
              int dt, int accumulate) {
  const int vec = vec_class(out, ld, elem_size(dt));
  A.job[A.n++] = Join{part, out, rows, cols, ld_part, ld, *grid, splits, vec, accumulate, dt};
  *grid += ceil_div(threads_of(rows, cols, kJoinCols, vec == 0), kElemThreads);
}

template <int DT, int ACT, int NT>
cudaError_t launch_few_of(const FewArgs& F, bool vec, cudaStream_t s) {
  const dim3 grid((unsigned)ceil_div(F.A.inner, kFewCols), (unsigned)ceil_div(F.A.rows, 8 * NT));
  return vec ? launch_dependent(few_kernel<DT, ACT, NT, true>, grid, dim3(kFewThreads), 0, s, F)
             : launch_dependent(few_kernel<DT, ACT, NT, false>, grid, dim3(kFewThreads), 0, s, F);
}
template <int DT, int ACT>
cudaError_t launch_few_act(const FewArgs& F, cudaStream_t s) {
  const bool vec = tma_ready(F.x, F.ld_x) && tma_ready(F.w[0], F.ld_w[0]) && tma_ready(F.w[1], F.ld_w[1]) && F.A.width % 8 == 0;
  return F.A.rows <= 8 ? launch_few_of<DT, ACT, 1>(F, vec, s) : launch_few_of<DT, ACT, 2>(F, vec, s);
}
cudaError_t launch_few(const FewArgs& F, int dt, cudaStream_t s) {
  auto of = [&](auto type) {
    constexpr int DT = decltype(type)::value;
    if (F.A.part || F.A.act == QMUON_ACT_SILU) return launch_few_act<DT, QMUON_ACT_SILU>(F, s);
    return F.A.act == QMUON_ACT_GELU ? launch_few_act<DT, QMUON_ACT_GELU>(F, s) : launch_few_act<DT, QMUON_ACT_GELU_TANH>(F, s);
  };
  return dt == QMUON_BF16 ? of(std::integral_constant<int, QMUON_BF16>{}) : of(std::integral_constant<int, QMUON_FP16>{});
}

// dh's maxima, of at most `most` CTAs; their number in A.
cudaError_t launch_dh_max(GemmArgs& A, uint32_t* out, int most, cudaStream_t s) {
  const bool any = A.vec_dh == 0;
  const int64_t threads = threads_of(A.rows, A.inner, kMaxCols, any);
  A.dh_max = out;
  A.dh_parts = (int32_t)std::min<int64_t>(most, ceil_div(threads, kMaxThreads * kMaxUnroll));
  const MaxArgs M{A.dh, A.rows, A.inner, A.ld_dh, threads, A.vec_dh, out};
  return launch_dependent(any ? dh_max_kernel<true> : dh_max_kernel<false>, dim3((unsigned)A.dh_parts), dim3(kMaxThreads), 0, s, M);
}

// The operands as the tensor maps read them: the caller's arrays, or aligned copies in the workspace.
cudaError_t bring_operands(const Geometry& G, unsigned char* ws, const void** x, int64_t* ld_x, const uint8_t* x_scale,
                           const void* (&w)[2], int64_t (&ld_w)[2], int64_t rows, int64_t width, int64_t inner, int dt, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  Repack jobs[3];
  int n = 0;
  if (G.copy_x) {
    void* to = ws + G.x;
    if (x_scale) e = launch_decode(static_cast<const uint8_t*>(*x), x_scale, to, rows, width, G.ld_x, dt, s);
    else jobs[n++] = Repack{static_cast<const uint16_t*>(*x), static_cast<uint16_t*>(to), *ld_x, G.ld_x, rows, width};
    *x = to;
    *ld_x = G.ld_x;
  }
  for (int i = 0; i < 2; ++i)
    if (G.copy_w[i]) {
      jobs[n++] = Repack{static_cast<const uint16_t*>(w[i]), reinterpret_cast<uint16_t*>(ws + G.w[i]), ld_w[i], G.ld_wp, inner, width};
      w[i] = ws + G.w[i];
      ld_w[i] = G.ld_wp;
    }
  return e == cudaSuccess ? launch_repack(jobs, n, s) : e;
}

constexpr int64_t kMaxDim = (int64_t)1 << 28;

bool sizes_ok(int64_t rows, int64_t width, int64_t inner) {
  // products of sizes stay within what the grids and the 32-bit unit counts hold
  return rows >= 0 && rows <= kMaxDim && width >= 1 && width <= kMaxDim && inner >= 1 && inner <= kMaxDim &&
         inner <= ((int64_t)1 << 36) / width && (rows == 0 || inner <= ((int64_t)1 << 38) / rows) &&
         (rows == 0 || width <= ((int64_t)1 << 38) / rows);
}
bool matrix_ok(const void* p, int64_t ld, int64_t cols, int es) {
  return p && is_aligned(p, es) && ld >= cols && ld <= ((int64_t)1 << 36);
}
bool enums_ok(int act, int dtype, int saved) {
  return act >= QMUON_ACT_SILU && act <= QMUON_ACT_GELU_TANH && dtype >= QMUON_BF16 && dtype <= QMUON_FP32 && saved >= QMUON_SAVE_NONE &&
         saved <= QMUON_SAVE_MXFP8;
}

qmuon_status check_forward(const qmuon_gated_ffn* c) {
  if (!c || !sizes_ok(c->rows, c->width, c->inner) || !enums_ok(c->act, c->dtype, c->saved)) return QMUON_ERR_INVALID_ARGUMENT;
  if (c->dtype == QMUON_FP32) return QMUON_ERR_UNSUPPORTED;
  if (c->saved == QMUON_SAVE_MXFP8 && c->inner % QMUON_SCALE_BLOCK) return QMUON_ERR_UNSUPPORTED;
  if (c->rows == 0) return QMUON_OK;
  if (!matrix_ok(c->x, c->ld_x, c->width, 2) || !matrix_ok(c->w_gate, c->ld_w_gate, c->width, 2) ||
      !matrix_ok(c->w_up, c->ld_w_up, c->width, 2) || !matrix_ok(c->h, c->ld_h, c->inner, 2))
    return QMUON_ERR_INVALID_ARGUMENT;
  if (c->saved == QMUON_SAVE_SAME && (!matrix_ok(c->gate, c->ld_gate, c->inner, 2) || !matrix_ok(c->up, c->ld_up, c->inner, 2)))
    return QMUON_ERR_INVALID_ARGUMENT;
  if (c->saved == QMUON_SAVE_MXFP8 &&
      (!c->gate || !c->up || !is_aligned(c->gate, 16) || !is_aligned(c->up, 16) || !c->gate_scale || !c->up_scale))
    return QMUON_ERR_INVALID_ARGUMENT;
  return QMUON_OK;
}

qmuon_status check_backward(const qmuon_gated_ffn_grad* c) {
  if (!c || !sizes_ok(c->rows, c->width, c->inner) || !enums_ok(c->act, c->dtype, c->saved)) return QMUON_ERR_INVALID_ARGUMENT;
  if (c->dtype == QMUON_FP32) return QMUON_ERR_UNSUPPORTED;
  if (c->grad_dtype != c->dtype && c->grad_dtype != QMUON_FP32) return QMUON_ERR_INVALID_ARGUMENT;
  if (c->saved == QMUON_SAVE_MXFP8 && c->inner % QMUON_SCALE_BLOCK) return QMUON_ERR_UNSUPPORTED;
  if (c->x_scale && c->width % QMUON_SCALE_BLOCK) return QMUON_ERR_UNSUPPORTED;
  if ((c->dw_gate == nullptr) != (c->dw_up == nullptr)) return QMUON_ERR_INVALID_ARGUMENT;
  const int gs = elem_size(c->grad_dtype);
  if (c->dw_gate && (!matrix_ok(c->dw_gate, c->ld_dw_gate, c->width, gs) || !matrix_ok(c->dw_up, c->ld_dw_up, c->width, gs)))
    return QMUON_ERR_INVALID_ARGUMENT;
  if (!c->dx && !c->dw_gate && !c->h) return QMUON_ERR_INVALID_ARGUMENT;
  if (c->rows == 0) return QMUON_OK;
  if (!matrix_ok(c->dh, c->ld_dh, c->inner, 2)) return QMUON_ERR_INVALID_ARGUMENT;
  if (needs_weights(*c) && (!matrix_ok(c->w_gate, c->ld_w_gate, c->width, 2) || !matrix_ok(c->w_up, c->ld_w_up, c->width, 2)))
    return QMUON_ERR_INVALID_ARGUMENT;
  if (needs_x(*c) && (c->x_scale ? !c->x || !is_aligned(c->x, 16) : !matrix_ok(c->x, c->ld_x, c->width, 2)))
    return QMUON_ERR_INVALID_ARGUMENT;
  if (c->saved == QMUON_SAVE_SAME && (!matrix_ok(c->gate, c->ld_gate, c->inner, 2) || !matrix_ok(c->up, c->ld_up, c->inner, 2)))
    return QMUON_ERR_INVALID_ARGUMENT;
  if (c->saved == QMUON_SAVE_MXFP8 &&
      (!c->gate || !c->up || !is_aligned(c->gate, 16) || !is_aligned(c->up, 16) || !c->gate_scale || !c->up_scale))
    return QMUON_ERR_INVALID_ARGUMENT;
  if (c->dx && !matrix_ok(c->dx, c->ld_dx, c->width, 2)) return QMUON_ERR_INVALID_ARGUMENT;
  if (c->h && !matrix_ok(c->h, c->ld_h, c->inner, 2)) return QMUON_ERR_INVALID_ARGUMENT;
  return QMUON_OK;
}

}  // namespace
}  // namespace lm
}  // namespace qm

using namespace qm;
using namespace qm::lm;

extern "C" size_t qmuon_gated_ffn_workspace_size(const qmuon_gated_ffn* c) {
  if (check_forward(c) != QMUON_OK) return 0;
  if (c->rows == 0) return kWsHeader;
  const int sms = num_sms();
  return forward_geometry(*c, std::max(1, (sms > 0 ? sms : 152) / 2)).total;
}

extern "C" qmuon_status qmuon_gated_ffn_forward(const qmuon_gated_ffn* c, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("qmuon_gated_ffn_forward");
  return no_throw("qmuon_gated_ffn_forward", [&]() -> qmuon_status {
    const qmuon_status st = check_forward(c);
    if (st != QMUON_OK) return st;
    if (c->rows == 0) return QMUON_OK;
    if (!ws || !is_aligned(ws, 256)) return QMUON_ERR_INVALID_ARGUMENT;
    const int sms = num_sms();
    if (sms <= 0) return set_error_msg("qmuon_gated_ffn_forward: SM count query failed", QMUON_ERR_CUDA);
    const Geometry G = forward_geometry(*c, std::max(1, sms / 2));
    if (ws_bytes < G.total) return QMUON_ERR_WORKSPACE_TOO_SMALL;
    unsigned char* b = static_cast<unsigned char*>(ws);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    GemmArgs A{};
    const void *x = c->x, *w[2] = {c->w_gate, c->w_up};
    int64_t ld_x = c->ld_x, ld_w[2] = {c->ld_w_gate, c->ld_w_up};
    A.rows = c->rows, A.width = c->width, A.inner = c->inner;
    A.tiles_m = G.tiles_m, A.tiles_n = G.tiles_n, A.splits = G.splits;
    A.units = G.tiles_m * G.tiles_n * G.splits;
    A.h = c->h, A.ld_h = c->ld_h, A.vec_h = vec_class(c->h, c->ld_h, 2);
    A.gate = c->gate, A.up = c->up, A.ld_gate = c->ld_gate, A.ld_up = c->ld_up;
    A.gate_scale = c->gate_scale, A.up_scale = c->up_scale;
    A.vec_gate = c->saved == QMUON_SAVE_MXFP8 ? vec_class(c->gate, 32, 1) : vec_class(c->gate, c->ld_gate, 2);
    A.vec_up = c->saved == QMUON_SAVE_MXFP8 ? vec_class(c->up, 32, 1) : vec_class(c->up, c->ld_up, 2);
    A.act = c->act, A.saved = c->saved;
    A.hdr = reinterpret_cast<WsHeader*>(b);
    A.ld_part = G.ld_fwd;
    A.part = G.part ? reinterpret_cast<float*>(b + G.part) : nullptr;
    cudaError_t e;
    if (G.few) {
      e = launch_few(FewArgs{A, x, {w[0], w[1]}, ld_x, {ld_w[0], ld_w[1]}}, c->dtype, s);
    } else {
      e = launch_clear(A.hdr, s);
      if (e == cudaSuccess) e = bring_operands(G, b, &x, &ld_x, nullptr, w, ld_w, c->rows, c->width, c->inner, c->dtype, s);
      if (e != cudaSuccess) return set_error("qmuon_gated_ffn_forward (operands)", e);
      if (!encode_map(&A.a[0], x, c->rows, c->width, ld_x, c->dtype) ||
          !encode_map(&A.b[0], w[0], c->inner, c->width, ld_w[0], c->dtype) ||
          !encode_map(&A.b[1], w[1], c->inner, c->width, ld_w[1], c->dtype))
        return QMUON_ERR_CUDA;
      e = launch_projections<K_FWD>(A, G, c->dtype, s);
    }
    if (e == cudaSuccess && A.part) {
      ElemArgs E{};
      E.A = A;
      E.part = A.part;
      E.splits = G.splits;
      e = launch_elem<FROM_PART, false>(E, c->dtype, s);
    }
    return e == cudaSuccess ? QMUON_OK : set_error("qmuon_gated_ffn_forward (launch)", e);
  });
}

extern "C" size_t qmuon_gated_ffn_backward_workspace_size(const qmuon_gated_ffn_grad* c) {
  if (check_backward(c) != QMUON_OK) return 0;
  if (c->rows == 0) return kWsHeader;
  const int sms = num_sms();
  return backward_geometry(*c, std::max(1, (sms > 0 ? sms : 152) / 2)).total;
}

extern "C" qmuon_status qmuon_gated_ffn_backward(const qmuon_gated_ffn_grad* c, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("qmuon_gated_ffn_backward");
  return no_throw("qmuon_gated_ffn_backward", [&]() -> qmuon_status {
    const qmuon_status st = check_backward(c);
    if (st != QMUON_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (c->rows == 0) {   // no rows: the weights' gradients are zero
      if (c->dw_gate && !c->accumulate) {
        const size_t gs = elem_size(c->grad_dtype);
        e = cudaMemset2DAsync(c->dw_gate, c->ld_dw_gate * gs, 0, c->width * gs, c->inner, s);
        if (e == cudaSuccess) e = cudaMemset2DAsync(c->dw_up, c->ld_dw_up * gs, 0, c->width * gs, c->inner, s);
      }
      return e == cudaSuccess ? QMUON_OK : set_error("qmuon_gated_ffn_backward (memset)", e);
    }
    if (!ws || !is_aligned(ws, 256)) return QMUON_ERR_INVALID_ARGUMENT;
    const int sms = num_sms();
    if (sms <= 0) return set_error_msg("qmuon_gated_ffn_backward: SM count query failed", QMUON_ERR_CUDA);
    const Geometry G = backward_geometry(*c, std::max(1, sms / 2));
    if (ws_bytes < G.total) return QMUON_ERR_WORKSPACE_TOO_SMALL;
    unsigned char* b = static_cast<unsigned char*>(ws);
    const void *x = c->x, *w[2] = {c->w_gate, c->w_up};
    int64_t ld_x = c->ld_x, ld_w[2] = {c->ld_w_gate, c->ld_w_up};
    // the header is cleared by the first kernel that needs no wait, where there is one
    if (c->saved == QMUON_SAVE_NONE && !G.few) e = launch_clear(reinterpret_cast<WsHeader*>(b), s);
    const void* w_given[2] = {c->w_gate, c->w_up};
    if (e == cudaSuccess) e = bring_operands(G, b, &x, &ld_x, c->x_scale, w, ld_w, c->rows, c->width, c->inner, c->dtype, s);
    if (e != cudaSuccess) return set_error("qmuon_gated_ffn_backward (operands)", e);

    GemmArgs A{};
    A.rows = c->rows, A.width = c->width, A.inner = c->inner;
    A.dh = c->dh, A.ld_dh = c->ld_dh, A.vec_dh = vec_class(c->dh, c->ld_dh, 2);
    A.h = c->h, A.ld_h = c->ld_h, A.vec_h = c->h ? vec_class(c->h, c->ld_h, 2) : 0;
    A.dgate = b + G.dgate, A.dup = b + G.dup, A.ld_d = G.ld_d;
    A.act = c->act, A.saved = c->saved;
    A.hdr = reinterpret_cast<WsHeader*>(b);
    if (c->dtype == QMUON_FP16 && (c->dx || c->dw_gate)) e = launch_dh_max(A, reinterpret_cast<uint32_t*>(b + G.dh_max), 2 * G.pairs, s);
    if (e != cudaSuccess) return set_error("qmuon_gated_ffn_backward (launch)", e);
    ElemArgs E{};
    if (c->saved == QMUON_SAVE_NONE) {   // gate and up again
      A.tiles_m = G.tiles_m, A.tiles_n = G.tiles_n, A.splits = G.splits;
      A.units = G.tiles_m * G.tiles_n * G.splits;
      A.ld_part = G.ld_fwd;
      A.part = G.part ? reinterpret_cast<float*>(b + G.part) : nullptr;
      if (G.few) {
        e = launch_few(FewArgs{A, x, {w_given[0], w_given[1]}, ld_x, {c->ld_w_gate, c->ld_w_up}}, c->dtype, s);
      } else {
        if (!encode_map(&A.a[0], x, c->rows, c->width, ld_x, c->dtype) ||
            !encode_map(&A.b[0], w[0], c->inner, c->width, ld_w[0], c->dtype) ||
            !encode_map(&A.b[1], w[1], c->inner, c->width, ld_w[1], c->dtype))
          return QMUON_ERR_CUDA;
        e = launch_projections<K_BWD>(A, G, c->dtype, s);
      }
      if (e == cudaSuccess && A.part) {
        E.A = A;
        E.part = A.part;
        E.splits = G.splits;
        e = launch_elem<FROM_PART, true>(E, c->dtype, s);
      }
    } else {
      const bool mx = c->saved == QMUON_SAVE_MXFP8;
      E.A = A;
      E.gate = c->gate, E.up = c->up, E.gate_scale = c->gate_scale, E.up_scale = c->up_scale;
      E.ld_gate = c->ld_gate, E.ld_up = c->ld_up;
      E.clear = 1;
      E.vec_in = mx ? std::min(vec_class(c->gate, 32, 1), vec_class(c->up, 32, 1))
                    : std::min(vec_class(c->gate, c->ld_gate, 2), vec_class(c->up, c->ld_up, 2));
      e = mx ? launch_elem<FROM_MXFP8, true>(E, c->dtype, s) : launch_elem<FROM_SAME, true>(E, c->dtype, s);
    }
    if (e != cudaSuccess) return set_error("qmuon_gated_ffn_backward (launch)", e);
    if (!c->dx && !c->dw_gate) return QMUON_OK;

    const int64_t units_x = (int64_t)G.dx_m * G.dx_n * G.dx_splits, units_w = 2 * (int64_t)G.dw_m * G.dw_n * G.dw_splits;
    const int pairs = (int)std::min<int64_t>(units_x + units_w, G.pairs);
    A.tiles_m = G.dx_m, A.tiles_n = G.dx_n, A.splits = G.dx_splits;
    A.tiles_wm = G.dw_m, A.tiles_wn = G.dw_n, A.splits_w = G.dw_splits;
    A.units = (int32_t)units_x, A.units_w = (int32_t)units_w;
    // dW units: the pairs without a last unit of dx take as many as its K blocks are worth; the rest goes round
    {
      const int extra = (int)(units_x % pairs), few = pairs - extra;
      const int64_t cost_x = 2 * ceil_div(c->inner, kBK) / G.dx_splits, cost_w = std::max<int64_t>(1, ceil_div(c->rows, kBK) / G.dw_splits);
      const int64_t worth = extra ? std::min((cost_x + cost_w / 2) / cost_w, units_w / few) : 0;
      A.few_w = (int32_t)worth;
      A.rounds_w = (int32_t)((units_w - worth * few) / pairs);
    }
    A.dx = c->dx, A.ld_dx = c->ld_dx, A.vec_dx = vec_class(c->dx, c->ld_dx, 2);
    const int gs = elem_size(c->grad_dtype);
    A.dw[0] = c->dw_gate, A.dw[1] = c->dw_up, A.ld_dw[0] = c->ld_dw_gate, A.ld_dw[1] = c->ld_dw_up;
    A.vec_dw[0] = vec_class(c->dw_gate, c->ld_dw_gate, gs), A.vec_dw[1] = vec_class(c->dw_up, c->ld_dw_up, gs);
    A.dw_f32 = c->grad_dtype == QMUON_FP32, A.accumulate = c->accumulate != 0;
    A.ld_part = G.ld_w;
    A.part = G.part_x ? reinterpret_cast<float*>(b + G.part_x) : nullptr;
    A.part_w = G.part_w ? reinterpret_cast<float*>(b + G.part_w) : nullptr;
    if (!encode_map(&A.a[0], A.dgate, c->rows, c->inner, G.ld_d, c->dtype) ||
        !encode_map(&A.a[1], A.dup, c->rows, c->inner, G.ld_d, c->dtype))
      return QMUON_ERR_CUDA;
    if (c->dx && (!encode_map(&A.b[0], w[0], c->inner, c->width, ld_w[0], c->dtype) ||
                  !encode_map(&A.b[1], w[1], c->inner, c->width, ld_w[1], c->dtype)))
      return QMUON_ERR_CUDA;
    if (c->dw_gate && !encode_map(&A.b[2], x, c->rows, c->width, ld_x, c->dtype)) return QMUON_ERR_CUDA;
    e = launch_gradients(A, units_x + units_w, pairs, c->dtype, s);
    JoinArgs J{};
    int64_t grid = 0;
    if (A.part) add_join(J, &grid, A.part, G.dx_splits, c->rows, c->width, G.ld_w, c->dx, c->ld_dx, c->dtype, 0);
    for (int i = 0; i < 2 && A.part_w; ++i)
      add_join(J, &grid, A.part_w + (size_t)i * G.dw_splits * c->inner * G.ld_w, G.dw_splits, c->inner, c->width, G.ld_w, A.dw[i], A.ld_dw[i],
               c->grad_dtype, A.accumulate);
    if (e == cudaSuccess && J.n) e = launch_dependent(join_kernel, dim3((unsigned)grid), dim3(kElemThreads), 0, s, J);
    return e == cudaSuccess ? QMUON_OK : set_error("qmuon_gated_ffn_backward (launch)", e);
  });
}
