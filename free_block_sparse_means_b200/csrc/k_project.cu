// Matrix product with its epilogue (sparsepr_project in include/sparsepr.h):
//   Y = R + gate_b * act(X W^T + bias)
// with X, Y and R row-major or head-major.  Two forms:
//
// k_project_few   At most FEW_ROWS rows: every weight is read once and used for
//   a handful of rows, so the bound is reading W.  A warp streams 8 rows of W
//   per load instruction straight into the B fragments of mma.sync (16 x 8 x 16,
//   the rows of X are A); the warps of a block split K and add up in shared memory.
//   4 rows x 5,120 x 5,120: 17.6 us, 3.0 TB/s of weights; x 20,480: 46.6 us, 4.5 TB/s.
//   (32 rows this way: 38 us at 5,120 x 5,120, the other form 22 us.)
//
// k_project_pair  Everything else, on the 5th-generation tensor cores.  Two CTAs
//   of a cluster make one tile of 256 rows x bn channels (cta_group::2): each
//   loads its 128 rows of X and half of the bn rows of W by TMA, a thread of the
//   first CTA issues the products of both, and each CTA keeps 128 x bn sums in
//   its TMEM, twice, so that the epilogue of one tile runs under the products of
//   the next.  Sharing W between the pair halves its traffic from L2, which a
//   128 x 256 tile per CTA is bound by.
//   A CTA: warp 0 loads into a ring of NST stages of 64 channels, warp 1 issues,
//   warps 4-11 are the epilogue (two warpgroups, 64 channels in turn each).  R comes
//   and Y leaves by TMA, which clips ragged edges and finds the head-major places.
//   Head-major X: 64 channels of K never cross a head (dx is a multiple of 64).
//   Rows: a tile's 128 rows are of one batch, or of several whole batches of at
//   most 64 rows (the box of the tensor map spans them).
//   75,600 x 5,120 x 5,120 with gate and residual, inputs changing: 3.02 to 3.14 ms at
//   1.15 to 1.25 GHz, 1,270 to 1,310 TFLOP/s; the tensor pipe is busy 0.89 of the time at
//   18,944 rows, so the power limit is the bound.  8,190 x 2,048 x 6,144 (768 tiles on 74
//   pairs, 10.4 rounds): 162 to 168 us at 1.4 GHz, 1,250 TFLOP/s.  Under `lane == 0` instead
//   of a uniform loop the issuing thread was the bound (12 % and 20 % longer).
//   With few stages to a tile the epilogue is the bound: 65,144 x 344 x 4,360 with bias and
//   silu (two operations of the multi-function unit an output) 390 us, without silu 334.
//   Where tiles are too few for the SMs, K is split, the sums go to the workspace
//   in fp32 and k_project_join adds them and does the epilogue.
//
// Every mbarrier wait is bounded, as in the routed attention kernel.
#include <cuda_fp16.h>

#include "tc_sm100.cuh"

namespace spr {
namespace {

constexpr int FEW_ROWS = 16;
constexpr int PBM = 128;                       // rows of a CTA's half of a tile
constexpr int PBK = 64;                        // channels of a stage: one swizzled 128-byte row
constexpr uint32_t PBOX = PBM * 128;           // 16 KB: 128 rows of 64 channels
constexpr int NST = 5;                         // stages, each X box and W box
constexpr int PJ_THREADS = 384;
constexpr uint32_t PJ_TMEM = 512;              // two accumulators of 256 columns
constexpr uint64_t PJ_WAIT_NS = 2000000000ull;  // 2 s
constexpr size_t PJ_SMEM = 1024 + (size_t)(2 * NST + 4) * PBOX + 256;
constexpr int MAX_SPLIT = 8;
constexpr size_t WORDS_BYTES = 256;  // of the workspace, before the splits' sums

// Division of 0 <= n < 2^31 by a fixed 1 <= d <= 2^31: with 2^s >= d and m = floor(2^(31 + s) / d) + 1,
// n m >> (31 + s) is exact, as m d - 2^(31 + s) <= d <= 2^s (Granlund and Montgomery).  A tile's
// place takes ten divisions, which cost its epilogue as much as its arithmetic.
struct FastDiv {
  uint32_t d, m, s;
  void set(uint32_t by) {
    d = by;
    s = 0;
    while ((1ull << s) < by) ++s;
    m = (uint32_t)((1ull << (31 + s)) / by + 1);
  }
  __device__ __forceinline__ int div(int n) const {
    return (int)((uint64_t)(uint32_t)n * m >> (31 + s));
  }
};

struct PjArgs {
  const void *X, *W, *bias, *gate, *R;
  void* Y;
  int64_t xs[3], ys[3], rs[3], ws;
  int B, N, K, M, dx, dy, act;
  int gate_rows;  // rows of a batch where the batches are taken as one (else 0)
  // the pair kernel's plan
  int bn, nb, row_tiles, tiles_per_batch, row_pairs, col_tiles, nsplit, kchunks, n_items;
  int share;  // stages of a split
  // by the splits, the tiles of a block of row pairs, the row pairs of the last block, a
  // batch's row tiles, dx and dy
  FastDiv by_split, by_group, by_last, by_batch, by_dx, by_dy;
  uint32_t x_bytes, r_bytes;  // of one box
  int xmul_b, xmul_h, ymul_b, ymul_h, rmul_b, rmul_h;  // 0 where a TMA dimension has one entry
  float* part;
  int32_t *status, *words;  // the call's, and the error words of its workspace
};

__device__ __forceinline__ float tof(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float tof(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ uint32_t pair_of(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pair_of<bf16>(float lo, float hi) { return pack_bf16(lo, hi); }
template <>
__device__ __forceinline__ uint32_t pair_of<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const T* t = reinterpret_cast<const T*>(&u[i]);
    f[2 * i] = tof(t[0]);
    f[2 * i + 1] = tof(t[1]);
  }
}

__device__ __forceinline__ float recip(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// x / (1 + e^-t).  The exponential's relative error grows with |t|, but where t is
// far below zero the quotient is small against x by e^t: |t| e^t 2^-24 <= 2^-25 of x.
__device__ __forceinline__ float gated(float x, float t) {
  return x * recip(1.f + ex2(-1.4426950408889634f * t));
}
template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if (ACT == SPR_ACT_GELU) return 0.5f * x * (1.f + erff(x * 0.70710678118654752f));
  if (ACT == SPR_ACT_GELU_TANH)  // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
    return gated(x, 1.5957691216057308f * fmaf(0.044715f * x * x, x, x));
  if (ACT == SPR_ACT_SILU) return gated(x, x);
  return x;
}

// gate_b act(sum + bias) of 8 neighbouring channels, `bias` and `gate` at the first of them or null
template <typename T, int ACT>
__device__ __forceinline__ void finish8(float* f, const T* bias, const T* gate) {
  if (bias) {
    float c[8];
    unpack8<T>(*reinterpret_cast<const uint4*>(bias), c);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += c[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = activate<ACT>(f[i]);
  if (gate) {
    float c[8];
    unpack8<T>(*reinterpret_cast<const uint4*>(gate), c);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= c[i];
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pair_of<T>(f[0], f[1]), pair_of<T>(f[2], f[3]), pair_of<T>(f[4], f[5]),
                    pair_of<T>(f[6], f[7]));
}
// op(f, c) of 64 neighbouring channels from `col` on, c the row `p` of M values.  Channels
// behind the last (of a ragged tile: clipped when it is stored) take some others' values.
template <typename T, typename Op>
__device__ __forceinline__ void each8(float* f, const T* p, int col, int M, Op op) {
  uint4 c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    c[j] = *reinterpret_cast<const uint4*>(p + min(col + 8 * j, M - 8));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float g[8];
    unpack8<T>(c[j], g);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[8 * j + i] = op(f[8 * j + i], g[i]);
  }
}
// `f` with the activation as a compile-time constant
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if (act == SPR_ACT_NONE)
    f(std::integral_constant<int, SPR_ACT_NONE>{});
  else if (act == SPR_ACT_GELU)
    f(std::integral_constant<int, SPR_ACT_GELU>{});
  else if (act == SPR_ACT_GELU_TANH)
    f(std::integral_constant<int, SPR_ACT_GELU_TANH>{});
  else
    f(std::integral_constant<int, SPR_ACT_SILU>{});
}

// ------------------------------------------------------------------ few rows
// Not through the read-only path (.nc): the kernel is resident before the one that may have
// written the weights ends.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
template <typename T>
__device__ __forceinline__ void mma_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_16816<bf16>(float* d, const uint32_t* a, uint32_t b0,
                                                uint32_t b1) {
  mma16816(d, a, b0, b1);
}
template <>
__device__ __forceinline__ void mma_16816<__half>(float* d, const uint32_t* a, uint32_t b0,
                                                  uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int FEW_WARPS = 16;  // of a block, at most

// A step: lane (g, q) holds 16 bytes, channels 8 q .. 8 q + 7, of row g of each
// operand.  Taken as the fragments of two products (words 0, 1 and 2, 3) they
// number the 32 channels in another order, the same one for X and W.
// NG groups of 8 rows of X (the second is the lower half of A), NT groups of 8
// rows of W, U steps in flight.
template <typename T, int NG, int NT, int U>
__global__ void __launch_bounds__(32 * FEW_WARPS) k_project_few(const __grid_constant__ PjArgs a) {
  constexpr int OUT = 8 * NT;  // channels of a block
  __shared__ float sums[FEW_WARPS][8 * NG][OUT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int warps = blockDim.x >> 5;
  after_previous();
  const int m0 = blockIdx.x * OUT, rows = a.B * a.N;
  const T* w[NT];
  bool has_w[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int m = m0 + 8 * j + g;
    has_w[j] = m < a.M;
    w[j] = static_cast<const T*>(a.W) + (int64_t)(has_w[j] ? m : 0) * a.ws;
  }
  const T* x[NG];
  bool has_x[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int t = 8 * i + g;
    has_x[i] = t < rows;
    const int b = has_x[i] ? t / a.N : 0, n = has_x[i] ? t % a.N : 0;
    x[i] = static_cast<const T*>(a.X) + b * a.xs[0] + (int64_t)n * a.xs[2];
  }
  float acc[NT][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // this lane's channel and its place in X: head by head
  int k = warp * 32 + 8 * q, kx = k;
  int64_t head = 0;
  while (k - 8 * q < a.K) {
    uint4 wv[U][NT], xv[U][NG];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = k < a.K;
#pragma unroll
      for (int j = 0; j < NT; ++j) wv[u][j] = in && has_w[j] ? ld_stream(w[j] + k) : zero;
      if (in)
        while (kx >= a.dx) {
          kx -= a.dx;
          head += a.xs[1];
        }
#pragma unroll
      for (int i = 0; i < NG; ++i)
        xv[u][i] = in && has_x[i] ? *reinterpret_cast<const uint4*>(x[i] + head + kx) : zero;
      k += 32 * warps;
      kx += 32 * warps;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint4 lo = xv[u][0], hi = NG > 1 ? xv[u][NG - 1] : zero;
      const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mma_16816<T>(acc[j], a0, wv[u][j].x, wv[u][j].y);
        mma_16816<T>(acc[j], a1, wv[u][j].z, wv[u][j].w);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 2 * NG; ++e)
      sums[warp][g + 8 * (e >> 1)][8 * j + 2 * q + (e & 1)] = acc[j][e];
  __syncthreads();
  for (int i = threadIdx.x; i < rows * OUT; i += blockDim.x) {
    const int t = i / OUT, c = i % OUT, m = m0 + c;
    if (m >= a.M) continue;
    float v = 0.f;
    for (int s = 0; s < warps; ++s) v += sums[s][t][c];
    if (a.bias) v += tof(static_cast<const T*>(a.bias)[m]);
    with_act(a.act, [&](auto act) { v = activate<decltype(act)::value>(v); });
    const int b = t / a.N, n = t % a.N, h = m / a.dy, ch = m - h * a.dy;
    if (a.gate) v *= tof(static_cast<const T*>(a.gate)[(int64_t)b * a.M + m]);
    if (a.R)
      v += tof(static_cast<const T*>(a.R)[b * a.rs[0] + h * a.rs[1] + (int64_t)n * a.rs[2] + ch]);
    const uint32_t one = pair_of<T>(v, v);
    reinterpret_cast<uint16_t*>(a.Y)[b * a.ys[0] + h * a.ys[1] + (int64_t)n * a.ys[2] + ch] =
        (uint16_t)one;
  }
}

// ------------------------------------------------------------ pairs of CTAs
// Row tile t: its first batch and row.
__device__ __forceinline__ void row_tile(const PjArgs& a, int t, int& b, int& n) {
  b = a.nb > 1 ? t * a.nb : a.by_batch.div(t);
  n = a.nb > 1 ? 0 : (t - b * a.tiles_per_batch) * PBM;
}
// Item: blocks of 8 row pairs, channel tile by channel tile, so that the tiles
// at work at one time share X and W in L2.
constexpr int GROUP = 8;
struct PjItem {
  int rp, ct, k0, k1, split;
  __device__ PjItem(const PjArgs& a, int item) {
    const int t = a.by_split.div(item), group = a.by_group.div(t);
    split = item - t * a.nsplit;
    const int in = t - group * (GROUP * a.col_tiles), rows = min(GROUP, a.row_pairs - group * GROUP);
    ct = rows == GROUP ? in / GROUP : a.by_last.div(in);
    rp = group * GROUP + in - ct * rows;
    const int share = a.share;
    k0 = min(split * share, a.kchunks);
    k1 = min(k0 + share, a.kchunks);
  }
};

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PJ_THREADS, 1)
    k_project_pair(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmR,
                   const __grid_constant__ PjArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sX = base;
  uint8_t* sW = base + NST * PBOX;
  uint8_t* sY = base + 2 * NST * PBOX;  // two buffers for each epilogue warpgroup
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + (2 * NST + 4) * PBOX);
  uint64_t* full = bars;                  // [NST] the first CTA's: both CTAs' loads
  uint64_t* empty = bars + NST;           // [NST]
  uint64_t* acc_full = bars + 2 * NST;    // [2]
  uint64_t* acc_empty = bars + 2 * NST + 2;  // [2] the first CTA's: both CTAs' epilogue warps
  uint64_t* r_full = bars + 2 * NST + 4;  // [2] R of each warpgroup
  uint64_t* drain = bars + 2 * NST + 6;
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(bars + 2 * NST + 7);
  volatile int* abort_s = reinterpret_cast<volatile int*>(tmem_base_s + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)tc::cluster_rank();
  const int first_item = blockIdx.x >> 1, step = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      tc::mbar_init(full + s, 1);
      tc::mbar_init(empty + s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(acc_full + s, 1);
      tc::mbar_init(acc_empty + s, 16);
      tc::mbar_init(r_full + s, 1);
    }
    tc::mbar_init(drain, 1);
    *abort_s = 0;
    tc::fence_barrier_init();
  }
  if (warp == 2) {
    tc::tmem_alloc_pair(tmem_base_s, PJ_TMEM);
    tc::tmem_relinquish_pair();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::tc_fence_after();
  const uint32_t tbase = *tmem_base_s;
  after_previous();

  if (warp == 0) {
    // -------------------------------------------------------------- loads
    if (lane == 0) {
      tc::prefetch_tmap(&tmX);
      tc::prefetch_tmap(&tmW);
      const uint32_t w_bytes = (uint32_t)a.bn * 64u;  // bn / 2 rows of 128 bytes
      int c = 0;
      bool ok = true;
      for (int w = first_item; w < a.n_items && ok; w += step) {
        const PjItem it(a, w);
        int b, n;
        row_tile(a, 2 * it.rp + rank, b, n);
        const int wrow = it.ct * a.bn + rank * (a.bn >> 1);
        int h = a.by_dx.div(it.k0 * PBK), x = it.k0 * PBK - h * a.dx;
        for (int k = it.k0; k < it.k1; ++k, ++c) {
          const int s = c % NST;
          if (c >= NST &&
              !(ok = tc::mbar_wait(empty + s, ((c / NST) - 1) & 1, abort_s, PJ_WAIT_NS)))
            break;
          if (rank == 0) tc::mbar_expect_tx(full + s, 2 * (a.x_bytes + w_bytes));
          const uint32_t bar = tc::leader_addr(full + s);
          tc::tma_load_4d_pair(sX + s * PBOX, &tmX, x, n, h * a.xmul_h, b * a.xmul_b, bar);
          tc::tma_load_2d_pair(sW + s * PBOX, &tmW, k * PBK, wrow, bar);
          if ((x += PBK) >= a.dx) x = 0, ++h;
        }
      }
      if (rank == 0 && *abort_s)  // let the pair's copies in flight land before it exits
        for (int k = c - NST; k < c; ++k)
          if (k >= 0) tc::mbar_wait_bounded(full + k % NST, (k / NST) & 1, 100000000ull);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- products
    // All lanes of the first CTA's warp run the loop, one issues: the operands
    // then come from uniform registers.
    if (rank == 0) {
      const uint32_t id = std::is_same<T, bf16>::value ? tc::idesc_bf16(2 * PBM, a.bn, 0)
                                                       : tc::idesc_fp16(2 * PBM, a.bn, 0);
      const uint64_t xd = tc::smem_desc_sw128(smem_u32(sX), 16, 1024);
      const uint64_t wd = tc::smem_desc_sw128(smem_u32(sW), 16, 1024);
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool got = tc::mbar_wait(bar, parity, abort_s, PJ_WAIT_NS);
        return __all_sync(0xffffffffu, got) != 0;
      };
      int c = 0, t = 0;
      bool ok = true;
      for (int w = first_item; w < a.n_items && ok; w += step) {
        const PjItem it(a, w);
        if (it.k0 == it.k1) continue;
        const uint32_t d = tbase + (t & 1) * 256;
        if (t >= 2 && !(ok = wait(acc_empty + (t & 1), ((t >> 1) - 1) & 1))) break;
        tc::tc_fence_after();
        uint32_t more = 0;  // the tile's first product starts its sums
        for (int k = it.k0; k < it.k1; ++k, ++c) {
          const int s = c % NST;
          if (!(ok = wait(full + s, (c / NST) & 1))) break;
          tc::tc_fence_after();
          const uint64_t at = (uint64_t)(s * (PBOX >> 4));
          if (tc::elect_one()) {
#pragma unroll
            for (int i = 0; i < PBK / 16; ++i)
              tc::mma_ss_pair(d, xd + at + 2 * i, wd + at + 2 * i, id, i > 0 ? 1u : more);
            tc::mma_commit_pair(empty + s);
            if (k + 1 == it.k1) tc::mma_commit_pair(acc_full + (t & 1));
          }
          __syncwarp();
          more = 1;
        }
        if (!ok) break;
        ++t;
      }
      if (tc::elect_one()) tc::mma_commit_pair(drain);
      __syncwarp();
      tc::mbar_wait_bounded(drain, 0, PJ_WAIT_NS);
    }
  } else if (warp >= 4) {
    // ----------------------------------------------------------- epilogue
    const int wg = (warp - 4) >> 2, tid = threadIdx.x & 127, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    // With a residual the first buffer is Y's and the second R's; without, Y takes
    // them in turn.
    uint8_t *const buf0 = sY + 2 * wg * PBOX, *const buf1 = buf0 + PBOX;
    const bool staged = a.nsplit == 1;
    int t = 0, nr = 0, ny = 0;
    // After a wait that gave up a warp still goes through its items, without
    // loading or storing sums, so that the warpgroup's barriers stay matched.
    bool ok = true, r_ok = true;
    for (int w = first_item; w < a.n_items; w += step) {
      const PjItem it(a, w);
      int b, n;
      const int rt = 2 * it.rp + rank;
      row_tile(a, rt, b, n);
      const int cols = min(a.bn, a.M - it.ct * a.bn);  // channels of the tile that exist
      const bool live_tile = rt < a.row_tiles;
      const int rows = a.nb > 1 ? min(a.nb, a.B - b) * a.N : min(PBM, a.N - n);  // that exist
      // R of the 64 channels from `c0` on
      auto load_r = [&](int c0) {
        if (tid == 0 && r_ok) {
          const int col = it.ct * a.bn + c0, h = a.by_dy.div(col);
          tc::mbar_expect_tx(r_full + wg, a.r_bytes);
          tc::tma_load_4d(buf1, &tmR, col - h * a.dy, n, h * a.rmul_h, b * a.rmul_b, r_full + wg);
        }
      };
      const bool mine = live_tile && wg * 64 < cols;
      if (staged && mine && a.R) load_r(wg * 64);
      const bool any = it.k0 < it.k1;
      if (any && ok) {
        const bool got = tc::mbar_wait(acc_full + (t & 1), (t >> 1) & 1, abort_s, PJ_WAIT_NS);
        __syncwarp();
        ok = __all_sync(0xffffffffu, got);
        tc::tc_fence_after();
      }
      const uint32_t acc = tbase + lanes + (t & 1) * 256;
      auto release = [&]() {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(tc::leader_addr(acc_empty + (t & 1)));
      };
      const T *bias = static_cast<const T*>(a.bias), *gate = static_cast<const T*>(a.gate);
      if (gate) {  // the row's batch
        int gb = b;
        if (a.gate_rows) gb = min(n + row, a.N - 1) / a.gate_rows;
        if (a.nb > 1) gb = min(b + row / a.N, a.B - 1);
        gate += (int64_t)gb * a.M;
      }
      if (mine)
        for (int c0 = wg * 64; c0 < cols; c0 += 128) {
          uint32_t v[64];
          if (ok && any) {
            __syncwarp();
            tc::tmem_ld32(acc + c0, v);
            tc::tmem_ld32(acc + c0 + 32, v + 32);
            tc::tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) v[i] = 0u;
          }
          if (any && c0 + 128 >= cols) release();  // the sums are in registers
          const int col = it.ct * a.bn + c0;
          if (!staged) {  // sums to the workspace
            float* p = a.part + ((int64_t)it.split * a.row_tiles * PBM + (int64_t)rt * PBM + row) *
                                    a.M + col;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c0 + 4 * j < cols && row < rows)
                reinterpret_cast<uint4*>(p)[j] =
                    make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            continue;
          }
          // Each step over all 64 channels: a branch for every 8 of them cost more than
          // the arithmetic (1,650 cycles a chunk without any activation).  Before the waits for
          // the buffers, under which bias and gate are on their way (65,144 x 344 x 4,360 with
          // bias 346 -> 334 us).
          float* f = reinterpret_cast<float*>(v);
          if (bias) each8<T>(f, bias, col, a.M, [](float x, float c) { return x + c; });
          if (a.act != SPR_ACT_NONE)
            with_act(a.act, [&](auto act) {
#pragma unroll
              for (int i = 0; i < 64; ++i) f[i] = activate<decltype(act)::value>(f[i]);
            });
          if (gate) each8<T>(f, gate, col, a.M, [](float x, float c) { return x * c; });
          // the buffer's last store has left it
          if (tid == 0) {
            if (a.R)
              tc::bulk_wait_read<0>();
            else
              tc::bulk_wait_read<1>();
          }
          if (a.R) {
            // whatever became of the products, this load is in flight
            const bool got = r_ok && tc::mbar_wait_bounded(r_full + wg, nr & 1, PJ_WAIT_NS);
            __syncwarp();
            ++nr;
            r_ok = __all_sync(0xffffffffu, got);
            if (!r_ok) ok = false, *abort_s = 1;
          }
          tc::named_sync(1 + wg, 128);
          uint8_t* to = a.R || !(ny & 1) ? buf0 : buf1;
          ++ny;
          if (a.R) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float r[8];
              unpack8<T>(*reinterpret_cast<const uint4*>(buf1 + row * 128 + ((j ^ (row & 7)) << 4)),
                         r);
#pragma unroll
              for (int i = 0; i < 8; ++i) f[8 * j + i] += r[i];
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(to + row * 128 + ((j ^ (row & 7)) << 4)) = pack8<T>(f + 8 * j);
          tc::fence_proxy_async_smem();
          tc::named_sync(1 + wg, 128);
          if (tid == 0 && ok && !*abort_s) {
            const int h = a.by_dy.div(col);
            tc::tma_store_4d(&tmY, to, col - h * a.dy, n, h * a.ymul_h, b * a.ymul_b);
            tc::bulk_commit();
          }
          if (a.R && c0 + 128 < cols) load_r(c0 + 128);  // all threads have read this one's
        }
      if (any) {
        if (!mine) release();
        ++t;
      }
    }
    if (tid == 0) tc::bulk_wait();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::tc_fence_after();
  if (threadIdx.x == 0 && *abort_s) report_timeout(a.status, a.words);
  if (warp == 2) tc::tmem_dealloc_pair(tbase, PJ_TMEM);
}

// The splits' sums of 8 channels of a row, in their order, and the epilogue.
template <typename T>
__global__ void __launch_bounds__(256) k_project_join(const __grid_constant__ PjArgs a) {
  after_previous();
  const int units = a.M / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.B * a.N * units) return;
  const int64_t r = i / units;
  const int m = (int)(i % units) * 8, b = (int)(r / a.N), n = (int)(r % a.N);
  const int64_t slot = a.nb > 1 ? (int64_t)(b / a.nb) * PBM + b % a.nb * a.N + n
                                : (int64_t)b * a.tiles_per_batch * PBM + n;
  float f[8] = {};
  for (int s = 0; s < a.nsplit; ++s) {
    const float4* p = reinterpret_cast<const float4*>(
        a.part + ((int64_t)s * a.row_tiles * PBM + slot) * a.M + m);
    const float4 u = p[0], v = p[1];
    f[0] += u.x; f[1] += u.y; f[2] += u.z; f[3] += u.w;
    f[4] += v.x; f[5] += v.y; f[6] += v.z; f[7] += v.w;
  }
  const T *bias = static_cast<const T*>(a.bias), *gate = static_cast<const T*>(a.gate);
  const int64_t gb = a.gate_rows ? n / a.gate_rows : b;
  with_act(a.act, [&](auto act) {
    finish8<T, decltype(act)::value>(f, bias ? bias + m : nullptr,
                                     gate ? gate + gb * a.M + m : nullptr);
  });
  const int h = m / a.dy, ch = m - h * a.dy;
  if (a.R) {
    float c[8];
    unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.R) + b * a.rs[0] +
                                               h * a.rs[1] + (int64_t)n * a.rs[2] + ch), c);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += c[e];
  }
  *reinterpret_cast<uint4*>(static_cast<T*>(a.Y) + b * a.ys[0] + h * a.ys[1] +
                            (int64_t)n * a.ys[2] + ch) = pack8<T>(f);
}

// --------------------------------------------------------------------- host
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Rows on 16 bytes; one place per element for an output.  Tokens that share a
// row (a token stride of 0) cannot be described to the TMA and are refused.
bool strides_fit(const int64_t* s, int B, int H, int N, bool out) {
  const int size[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    if (s[i] < 0 || (size[i] > 1 && s[i] % 8)) return false;
    if (size[i] > 1 && s[i] == 0 && (out || i == 2)) return false;
  }
  return true;
}

spr_status check(const spr_project_params* p) {
  if (!p) return SPR_EINVAL;
  if (p->B < 1 || p->N < 1 || p->Hx < 1 || p->dx < 1 || p->Hy < 1 || p->dy < 1) return SPR_EINVAL;
  if (p->dtype != SPR_BF16 && p->dtype != SPR_FP16) return SPR_EINVAL;
  if (p->act < SPR_ACT_NONE || p->act > SPR_ACT_SILU) return SPR_EINVAL;
  if (p->dx % 8 || p->dy % 8) return SPR_EUNSUPPORTED;
  if ((p->Hx > 1 && p->dx % 64) || (p->Hy > 1 && p->dy % 64)) return SPR_EUNSUPPORTED;
  const int64_t K = (int64_t)p->Hx * p->dx, M = (int64_t)p->Hy * p->dy;
  if (K > (1 << 20) || M > (1 << 20) || (int64_t)p->B * p->N > (1 << 30) || p->B > 65535)
    return SPR_EUNSUPPORTED;
  if (p->w_stride < 0 || (M > 1 && (p->w_stride % 8 || p->w_stride < K))) return SPR_EUNSUPPORTED;
  if (!strides_fit(p->x_strides, p->B, p->Hx, p->N, false) ||
      !strides_fit(p->y_strides, p->B, p->Hy, p->N, true))
    return SPR_EUNSUPPORTED;
  return SPR_OK;
}

// What a call does: fills the shape and the plan of `a`; the workspace in bytes.
size_t make_plan(const spr_project_params& p, int sms, PjArgs* a) {
  a->B = p.B;
  a->N = p.N;
  a->K = p.Hx * p.dx;
  a->M = p.Hy * p.dy;
  a->dx = p.dx;
  a->dy = p.dy;
  a->act = p.act;
  a->ws = p.w_stride;
  for (int i = 0; i < 3; ++i) {
    a->xs[i] = p.x_strides[i];
    a->ys[i] = p.y_strides[i];
    a->rs[i] = p.r_strides[i];
  }
  if ((int64_t)p.B * p.N <= FEW_ROWS) return WORDS_BYTES;
  // Batches that follow one another row by row are one batch.
  auto in_a_row = [&](const int64_t* s) { return s[0] == (int64_t)p.N * s[2]; };
  // (the residual's strides are the caller's or Y's: the plan and so the
  // workspace do not depend on whether a residual is given)
  if (p.B > 1 && p.N > 1 && in_a_row(a->xs) && in_a_row(a->ys) && in_a_row(a->rs)) {
    a->gate_rows = p.N;
    a->N = p.B * p.N;
    a->B = 1;
  }
  // Short batches share a row tile where the tensors' batches can be boxed.
  a->nb = 1;
  if (a->B > 1 && 2 * a->N <= PBM && a->xs[0] && a->rs[0])
    a->nb = a->B < PBM / a->N ? a->B : PBM / a->N;
  a->tiles_per_batch = (a->N + PBM - 1) / PBM;
  a->row_tiles = a->nb > 1 ? (a->B + a->nb - 1) / a->nb : a->B * a->tiles_per_batch;
  a->row_pairs = (a->row_tiles + 1) / 2;
  a->kchunks = (a->K + PBK - 1) / PBK;
  // Channels of a tile and splits of K with the least estimated time, in cycles,
  // from measured calls: a stage of 64 channels takes 200 + 1.7 bn (its products
  // 2 bn; below 256 channels its bytes from L2), all weights at least what HBM
  // takes for them; a tile costs 1,200 to change over; splits cost a second
  // launch and the sums' way out and back.  64 rows x 2,048 x 2,048: bn 256 16.9 us,
  // 192 14.8, 128 12.7, 128 in three splits 11.8; 700 rows: 18.0, 15.7, 14.0, 21.2.
  const int clusters = sms / 2;
  double best = 0;
  for (int bn = 256; bn >= 64; bn -= 64) {
    const int ct = (a->M + bn - 1) / bn;
    const int64_t tiles = (int64_t)a->row_pairs * ct;
    for (int s = 1; s <= MAX_SPLIT; ++s) {
      if (s > 1 && (tiles * s > clusters || a->kchunks < 4 * s)) break;
      const int64_t waves = (tiles * s + clusters - 1) / clusters;
      const int chunks = (a->kchunks + s - 1) / s;
      const double stages = (double)waves * (chunks * (200.0 + 1.7 * bn) + 1200.0);
      const double weights = 2.0 * a->M * a->K / 2100.0;
      const double cost = (stages > weights ? stages : weights) +
                          (s > 1 ? 7600.0 + 8.0 * s * a->B * a->N * a->M / 2600.0 : 0.0);
      if (best == 0 || cost < best) {
        best = cost;
        a->bn = bn;
        a->col_tiles = ct;
        a->nsplit = s;
        a->n_items = (int)(tiles * s);
      }
    }
  }
  a->share = (a->kchunks + a->nsplit - 1) / a->nsplit;
  a->by_split.set(a->nsplit);
  a->by_group.set(GROUP * a->col_tiles);
  a->by_last.set(a->row_pairs % GROUP ? a->row_pairs % GROUP : GROUP);
  a->by_batch.set(a->tiles_per_batch);
  a->by_dx.set(a->dx);
  a->by_dy.set(a->dy);
  return WORDS_BYTES + (a->nsplit > 1 ? (size_t)a->nsplit * a->row_tiles * PBM * a->M * 4 : 0);
}

// [B, H, N, d] as a TMA map of boxes of `rows` rows (of `batches` batches) of 64
// channels.  A dimension of stride 0 becomes one entry whose coordinate stays 0.
bool make_map(CUtensorMap* m, const void* ptr, CUtensorMapDataType dt, int B, int H, int N, int d,
              const int64_t* s, int rows, int batches, int* mul_b, int* mul_h) {
  *mul_b = B > 1 && s[0] ? 1 : 0;
  *mul_h = H > 1 && s[1] ? 1 : 0;
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)N, (uint64_t)(*mul_h ? H : 1),
                            (uint64_t)(*mul_b ? B : 1)};
  auto bytes = [&](int64_t st, bool on) { return on ? (uint64_t)st * 2 : (uint64_t)d * 2; };
  const uint64_t strides[3] = {bytes(s[2], N > 1), bytes(s[1], *mul_h), bytes(s[0], *mul_b)};
  for (uint64_t st : strides)
    if (st >> 40) return false;
  const uint32_t box[4] = {PBK, (uint32_t)rows, 1, (uint32_t)batches};
  return encode_tmap(m, dt, 4, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename T>
cudaError_t launch_pair(const PjArgs& a, const CUtensorMap& x, const CUtensorMap& w,
                        const CUtensorMap& y, const CUtensorMap& r, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(k_project_pair<T>, PJ_SMEM, done);
  if (e != cudaSuccess) return e;
  const int clusters = sms / 2 < a.n_items ? sms / 2 : a.n_items;
  spr_launch_early(k_project_pair<T>, 2 * clusters, PJ_THREADS, PJ_SMEM, st, x, w, y, r, a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.nsplit == 1) return e;
  const int64_t units = (int64_t)a.B * a.N * (a.M / 8);
  spr_launch_early(k_project_join<T>, (unsigned)((units + 255) / 256), 256, 0, st, a);
  return cudaGetLastError();
}

template <typename T, int NG, int NT, int U>
cudaError_t launch_few(const PjArgs& a, int sms, cudaStream_t st) {
  // Warps of a block: as many as make about 22 of them on every SM, each with a
  // few rounds of its U steps at least.
  const int blocks = (a.M + 8 * NT - 1) / (8 * NT), rounds = (a.K + 32 * U - 1) / (32 * U);
  int warps = (22 * sms + blocks / 2) / blocks;
  if (warps > rounds) warps = rounds;
  warps = warps < 4 ? 4 : warps > FEW_WARPS ? FEW_WARPS : warps;
  spr_launch_early(k_project_few<T, NG, NT, U>, blocks, 32 * warps, 0, st, a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_few(const PjArgs& a, int sms, cudaStream_t st) {
  // Steps in flight: more of them cost more in resident warps than they bring (4 rows x
  // 5,120 x 5,120: 2 steps 19.6 us, 3 16.6, 4 16.1, 6 25.2, 8 20.6; x 20,480: 53.9, 45.1,
  // 52.0, 50.8, 49.2).  9 to 16 rows take two groups of 8 rows of W, so that X is read
  // half as often (2 steps 16.5 us, 3 26.6, 4 31.2).
  return a.B * a.N <= 8 ? launch_few<T, 1, 1, 3>(a, sms, st) : launch_few<T, 2, 2, 2>(a, sms, st);
}

}  // namespace
}  // namespace spr

using namespace spr;

extern "C" size_t sparsepr_project_workspace(const spr_project_params* p) {
  PjArgs a{};
  return check(p) == SPR_OK ? make_plan(*p, num_sms(), &a) : 0;
}

extern "C" spr_status sparsepr_project(const spr_project_params* p, const void* X, const void* W,
                                       const void* bias, const void* gate, const void* R, void* Y,
                                       void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  const spr_status s = check(p);
  if (s != SPR_OK) return s;
  if (!X || !W || !Y) return SPR_EINVAL;
  const int sms = num_sms();
  PjArgs a{};
  const size_t need = make_plan(*p, sms, &a);
  if (!ws || !aligned(ws, 256) || ws_bytes < need) return SPR_EWORKSPACE;
  if (!aligned(X, 16) || !aligned(W, 16) || !aligned(Y, 16) || !aligned(R, 16) ||
      !aligned(bias, 16) || !aligned(gate, 16) || !aligned(status, 4))
    return SPR_EUNSUPPORTED;
  if (R && !strides_fit(p->r_strides, p->B, p->Hy, p->N, false)) return SPR_EUNSUPPORTED;
  a.X = X;
  a.W = W;
  a.bias = bias;
  a.gate = gate;
  a.R = R;
  a.Y = Y;
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + WORDS_BYTES);
  a.words = static_cast<int32_t*>(ws);
  a.status = status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool few = a.n_items == 0;
  CUtensorMap mx{}, mw{}, my{}, mr{};
  if (!few) {
    const CUtensorMapDataType dt = p->dtype == SPR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if (!tmap_available()) return SPR_ECUDA;
    const int rows = a.nb > 1 ? a.N : PBM;
    const uint64_t wdims[2] = {(uint64_t)a.K, (uint64_t)a.M};
    const uint64_t wstride[1] = {(uint64_t)(a.M > 1 ? a.ws : a.K) * 2};
    const uint32_t wbox[2] = {PBK, (uint32_t)(a.bn / 2)};
    if (!make_map(&mx, X, dt, a.B, p->Hx, a.N, p->dx, a.xs, rows, a.nb, &a.xmul_b, &a.xmul_h) ||
        !make_map(&my, Y, dt, a.B, p->Hy, a.N, p->dy, a.ys, rows, a.nb, &a.ymul_b, &a.ymul_h) ||
        !make_map(&mr, R ? R : Y, dt, a.B, p->Hy, a.N, p->dy, R ? a.rs : a.ys, rows, a.nb,
                  &a.rmul_b, &a.rmul_h) ||
        wstride[0] >> 40 ||
        !encode_tmap(&mw, dt, 2, W, wdims, wstride, wbox, CU_TENSOR_MAP_SWIZZLE_128B))
      return SPR_EUNSUPPORTED;
    a.x_bytes = a.r_bytes = (uint32_t)(rows * a.nb) * 128u;
  }
  if (status && cudaMemsetAsync(status, 0, 4 * sizeof(int32_t), st) != cudaSuccess)
    return SPR_ECUDA;
  cudaError_t e;
  if (p->dtype == SPR_BF16)
    e = few ? launch_few<bf16>(a, sms, st) : launch_pair<bf16>(a, mx, mw, my, mr, sms, st);
  else
    e = few ? launch_few<__half>(a, sms, st) : launch_pair<__half>(a, mx, mw, my, mr, sms, st);
  return e == cudaSuccess ? SPR_OK : SPR_ECUDA;
}
