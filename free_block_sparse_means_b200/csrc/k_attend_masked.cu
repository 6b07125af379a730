// Exact attention under a mask (sparsepr_attend_masked in include/sparsepr.h) on
// the 5th-generation tensor cores.
//
//   x_ij = cap(scale q_i . k_j) - slope |p_i - j|,  O_i = sum_j softmax_j(x_i) v_j
//
// over the keys a query sees.  One pass over the keys with the running maximum
// m and sum l of every row: S = Q K^T of a 128 x 128 tile lands in TMEM, the
// softmax warps turn it into P = 2^(x - m) in place, O += P V accumulates in
// TMEM, and O is rescaled only when a row's maximum grows by more than 2^8 (the
// final division uses the same stale m, so that is exact).
//
// A persistent CTA per SM has two streams of 128 query rows, each with its own
// S / P and O in TMEM (4 x 128 columns) and its own softmax warpgroup of one
// row per thread, so that one stream's products run under the other's softmax:
//   PAIR  the streams are two neighbouring 128-row tiles of a head; a K or V
//         tile in shared memory serves both.
//   SOLO  (at most 128 rows share the keys: few query tokens, the heads of a
//         key head packed into the tile's rows) both streams hold the same
//         rows and take the key tiles in turn.
// Roles: warps 0-3 and 4-7 the softmax of stream 0 and 1; warp 8 makes the work
// items, passes them on through a ring and loads K and V tiles by TMA into
// another; warp 9 issues every product.  Where the items do not fill the SMs
// the keys are split; streams then write (O, m, l) in fp32 and k_am_join adds
// them up.
//
// What bounds it: a 128 x 128 tile is 1,024 cycles of products (d = 128) and, at 16
// exponentials a cycle, 1,024 of the multi-function unit; two streams' tiles take
// 4,050 cycles on an SM, the tensor pipe busy 0.51 and the multi-function unit 0.62 of
// them by their counters.  The softmax's own chain (scores out of TMEM, maximum,
// exponentials, P back) is the longest part, so it is cut short: the exponentials go
// ahead with the old maximum, and the product with V starts on the first half of P.
// 16 heads x 16,384 x 16,384, d = 128, inputs changing: 2,070 to 2,110 us at 1.74 GHz,
// 1,050 TFLOP/s; d = 64: 1,715 us at 1.965 GHz, 640 TFLOP/s.
// Measured and not kept (same case, on one box where this form took 1,820 us):
// products issued under `lane == 0` 2,307 us; a quarter of the exponentials as
// polynomials on the FMA pipe 2,067; a row shared by two threads, 16 softmax warps
// 2,243; S, P and O in steps of 64 keys 2,449.
// SOLO is bound by reading K and V: 8 x 8 key heads, 12,950 to 32,768 keys: 165 to 175 us
// with the join, 4.8 TB/s.
//
// Masks: with causal and prefix a row sees exactly the keys below one limit,
// which grows with the row, so a tile is skipped, partly masked or whole by
// comparing two limits.  Documents are classified per (256 rows, 128 keys) by
// their id ranges in k_am_documents, which lists the tiles to visit.
// Keys that count for nobody (past the length or the last row's limit, negative
// document) have their V rows zeroed in shared memory before the product: 0 x NaN would be NaN.
//
// Every mbarrier wait is bounded, as in the routed attention kernel.
#include <cfloat>
#include <cuda_fp16.h>

#include "tc_sm100.cuh"

namespace spr {
namespace {

constexpr int TBM = 128, TBN = 128;  // query rows of a stream, keys of a tile
constexpr uint32_t BOX = TBN * 128;  // one swizzled box of 128 rows x 64 channels: 16 KB
constexpr int AM_THREADS = 384;      // two softmax warpgroups; a loading, an issuing and two idle warps
// Registers: 168 a thread at launch (64,512 in all); a softmax thread holds a row of 128 scores.
// 2 x 128 x 200 + 128 x 104 = 64,512.
constexpr int SOFTMAX_REGS = 200, OTHER_REGS = 104;
constexpr uint32_t TMEM_COLS = 512, O_COL = 256;  // S0 | S1 | O0 | O1, 128 columns each
constexpr uint64_t WAIT_NS = 2000000000ull;  // 2 s
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.69314718055994531f;

template <int D>
__host__ __device__ constexpr uint32_t tile_bytes() { return TBN * D * 2; }
template <int D>
__host__ __device__ constexpr int ring() { return D == 128 ? 5 : 8; }  // K and V tiles in flight
// (the last 1024: barriers and the ring of items)
template <int D>
__host__ __device__ constexpr size_t smem_bytes() {
  return 1024 + (2 + ring<D>()) * (size_t)tile_bytes<D>() + 1024;
}

struct AmArgs {
  void* O;
  float* lse;
  const int32_t *k_len, *doc_q, *doc_k, *prefix;
  const float* slopes;
  int64_t os[3];
  int o_wide;  // rows of O lie on 32 bytes
  int B, Hq, Hk, Nq, Nk, causal, q_start;
  int qmul_b, qmul_h, kmul_b, kmul_h, vmul_b, vmul_h;  // 0 where a TMA dimension has one entry
  float scale, softcap, kz;  // kz: scale / softcap
  // the plan: tiles of rows (heads packed per tile `pack`, query blocks `nqb`), key splits
  int pack, ntile_h, nqb, nsplit, n_items, by_block;
  int n_tiles, n_whole;  // row tiles; the first n_whole are one item each, the rest nsplit
  // workspace: per row tile its listed key tiles (documents), partial results
  const int32_t *doc_count, *doc_list;
  int* next_item;  // counter of the items taken, or null: a fixed share for each block
  int ktiles;
  float *part_o, *part_ml;
  int part_rows;  // rows of a row tile that partial results hold
  int32_t *status, *words;  // the call's, and the error words of its workspace
};

// What the mask leaves of one batch's keys for query rows first .. last: rows see
// the keys below limit(row), which does not decrease with the row.
struct Limits {
  int len, pre, pos0, causal;
  int end;  // keys from here on are seen by no row of the batch
  __device__ __forceinline__ void init(const AmArgs& a, int b) {
    len = a.k_len ? min(max(a.k_len[b], 0), a.Nk) : a.Nk;
    pre = a.prefix ? min(max(a.prefix[b], 0), len) : 0;
    pos0 = a.q_start == SPR_ALIGN_END ? len - a.Nq : a.q_start;
    causal = a.causal;
    end = limit(a.Nq - 1);
  }
  __device__ __forceinline__ int limit(int row) const {
    return causal ? max(min(pos0 + row + 1, len), pre) : len;
  }
  // The place of row's position among the keys 0 .. len - 1 or next to them.  For all of these keys
  // |p - j| = |p - near| + |near - j|: the first part, the same for all of a row's scores, is
  // left to its lse (beyond()), so that far positions cost the scores no bits.
  __device__ __forceinline__ int nearest(int row) const {
    return max(min(pos0 + row, len - 1), 0);
  }
  __device__ __forceinline__ float beyond(int row) const {
    return (float)abs(pos0 + row - nearest(row));
  }
};

// One work item: a row tile (or pair of them) and its share of the key tiles.  The
// loading thread makes it and passes it on through a ring in shared memory.
template <bool SOLO>
struct Item {
  int b, h0, q0;       // batch, first query head, first query row
  int n, i0;           // key tiles of the item (-1: no more items) and the first of them
  int nt[2];           // key tiles each stream visits, from key 0 on
  int last[2];         // entry after which a stream has no more tiles, at the latest
  int near;            // with a distance penalty: the tile of the rows' position, else -1
  int64_t part;        // its first partial result, or -1: it writes O
  const int32_t* list; // documents: the listed tiles
  Limits lim;
  // Row tile number `at`, in the order they are taken.
  __device__ __forceinline__ void place(const AmArgs& a, int at) {
    const int heads = a.B * a.ntile_h;
    const int blk = a.by_block ? at / heads : at % a.nqb, t = a.by_block ? at % heads : at / a.nqb;
    const int ht = t % a.ntile_h;
    b = t / a.ntile_h;
    // heads: `pack` query heads per tile within a key head
    const int rep = a.Hq / a.Hk, per = (rep + a.pack - 1) / a.pack;
    h0 = (ht / per) * rep + (ht % per) * a.pack;
    // blocks with the most keys first: later items then even out the SMs
    // (across all heads with by_block)
    q0 = (a.causal ? a.nqb - 1 - blk : blk) * (SOLO ? TBM : 2 * TBM);
  }
  __device__ void init(const AmArgs& a, int item) {
    const bool whole = item < a.n_whole;
    const int k = item - a.n_whole, ns = whole ? 1 : a.nsplit, split = whole ? 0 : k % ns;
    part = whole ? -1 : (int64_t)k * 2;
    place(a, whole ? item : a.n_whole + k / ns);
    lim.init(a, b);
    nt[0] = tiles(a, 0);
    nt[1] = SOLO ? nt[0] : tiles(a, 1);
    int most = max(nt[0], nt[1]);
    list = nullptr;
    // Nearest keys first: their scores are the highest, so the maximum seldom moves.
    near = a.slopes ? min(max((lim.pos0 + q0 + (SOLO ? 0 : TBM)) / TBN, -1), most - 1) : -1;
    for (int s = 0; s < 2; ++s) last[s] = nt[s] - 1 > near ? nt[s] - 1 : near;
    if (a.doc_q) {
      const int64_t row = (int64_t)b * a.nqb + q0 / (SOLO ? TBM : 2 * TBM);
      list = a.doc_list + row * a.ktiles;
      most = a.doc_count[4 * row];
      last[0] = a.doc_count[4 * row + 1];
      last[1] = a.doc_count[4 * row + 2];
    }
    const int share = (most + ns - 1) / ns;
    i0 = min(most, split * share);
    n = min(most, i0 + share) - i0;
    for (int s = 0; s < 2; ++s) last[s] = SOLO ? n - 1 : min(last[s] - i0, n - 1);
  }
  __device__ __forceinline__ int tiles(const AmArgs& a, int s) const {
    const int first = q0 + s * TBM, last = min(first + TBM, a.Nq) - 1;
    return first < a.Nq ? (lim.limit(last) + TBN - 1) / TBN : 0;
  }
  // entry i: key tile and bits (1, 2: stream 0, 1 visits it; 4, 8: whole for it by documents;
  // 16: holds keys that count for nobody)
  __device__ __forceinline__ int entry(int i, int& bits) const {
    if (list) {
      const int e = list[i0 + i];
      bits = e & 31;
      return e >> 5;
    }
    int t = i0 + i;
    if (t <= near) t = near - t;  // the rows' own tile first, then back, then on
    bits = 12 | (t < nt[0] ? 1 : 0) | (t < nt[1] ? 2 : 0) | ((t + 1) * TBN > lim.end ? 16 : 0);
    return t;
  }
  __device__ __forceinline__ uint32_t streams(int i) const {
    int bits;
    entry(i, bits);
    return bits & 3;
  }
};

constexpr int ITEMS = 4;  // items in the ring

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c) {
  asm("{\n.reg .b64 ra, rb, rc, rd;\n"
      "mov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %4};\nmov.b64 rc, {%5, %5};\n"
      "fma.rn.ftz.f32x2 rd, ra, rb, rc;\nmov.b64 {%0, %1}, rd;\n}\n"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1) {
  asm("{\n.reg .b64 ra, rd;\n"
      "mov.b64 ra, {%2, %3};\nmov.b64 rd, {%0, %1};\n"
      "add.rn.ftz.f32x2 rd, rd, ra;\nmov.b64 {%0, %1}, rd;\n}\n"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1));
}
// (a0, a1) * b + (c0, c1)
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c0,
                                     float c1) {
  asm("{\n.reg .b64 ra, rb, rc, rd;\n"
      "mov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %4};\nmov.b64 rc, {%5, %6};\n"
      "fma.rn.ftz.f32x2 rd, ra, rb, rc;\nmov.b64 {%0, %1}, rd;\n}\n"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
// (d0, d1) * (a0, a1) + c
__device__ __forceinline__ void fma2e(float& d0, float& d1, float a0, float a1, float c) {
  asm("{\n.reg .b64 ra, rc, rd;\n"
      "mov.b64 ra, {%2, %3};\nmov.b64 rc, {%4, %4};\nmov.b64 rd, {%0, %1};\n"
      "fma.rn.ftz.f32x2 rd, rd, ra, rc;\nmov.b64 {%0, %1}, rd;\n}\n"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1), "f"(c));
}
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n.reg .b64 ra, rb, rd;\n"
      "mov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %5};\n"
      "mul.rn.ftz.f32x2 rd, ra, rb;\nmov.b64 {%0, %1}, rd;\n}\n"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void store32(void* p, const uint32_t* u) {  // p on 32 bytes
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]),
               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<bf16>(float lo, float hi) { return pack_bf16(lo, hi); }
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The cap c tanh(z), z = x kz, kz = scale / c, of scores x, in units of log 2.  Where
// |z| <= 0.6 it is x times a polynomial in x^2: tanh(z) / z fitted in z^2 for least error
// (2^-23.4 relative, in exact arithmetic), with kz and the scale in its coefficients; 6
// packed operations for two scores, none on the multi-function unit.  (Working in z takes
// 7, as does a cap with a penalty: 2 x 16 heads x 4,097 x 4,097, d = 64, with a prefix, 272 us
// against 267.)  Beyond, it is
// c - 2 c / (1 + e^(2 z)), whose error is a few 2^-24 of c: near 0 that would be all of a
// score, so each score takes the form that is exact relative to itself.
// Z: in z, with coefficients of usual size under any cap.
template <bool Z>
struct Cap {
  float kz, c0, c1, c2, c3, c4, most;  // coefficients, and the largest x^2 (z^2) they hold for
  __device__ __forceinline__ void init(float scale, float cap, float ratio) {
    kz = ratio;
    const float k2 = Z ? 1.f : kz * kz;
    c0 = (Z ? cap : scale) * LOG2E;
    c1 = -0.33332622051239014f * k2 * c0;
    c2 = 0.13313521444797516f * k2 * k2 * c0;
    c3 = -0.05223110690712929f * k2 * k2 * k2 * c0;
    c4 = 0.01564048044383526f * k2 * k2 * k2 * k2 * c0;
    most = 0.36f / k2;
  }
};
// Whether a cap's coefficients (kz^9 c in c4) are normal fp32 numbers.
bool cap_is_usual(float scale, float cap) {
  const float kz = scale / cap;
  return kz >= 0x1p-12f && kz <= 0x1p8f && cap >= 0x1p-12f && cap <= 0x1p50f;
}
// x^2 (z^2) of two scores, and the polynomial's value
template <bool Z>
__device__ __forceinline__ void cap_poly(const float* x, float* u, float* y, const Cap<Z>& c) {
  float z0 = x[0], z1 = x[1], p0, p1;
  if (Z) mul2(z0, z1, x[0], x[1], c.kz, c.kz);
  mul2(u[0], u[1], z0, z1, z0, z1);
  fma2(p0, p1, u[0], u[1], c.c4, c.c3);
  fma2e(p0, p1, u[0], u[1], c.c2);
  fma2e(p0, p1, u[0], u[1], c.c1);
  fma2e(p0, p1, u[0], u[1], c.c0);
  mul2(y[0], y[1], z0, z1, p0, p1);
}
// Caps a tile's scores if all of a warp's are near; else false, with x spoiled.  Rows that
// are not `live` have no say: theirs come of whatever the shared memory behind packed rows held.
template <bool Z>
__device__ __forceinline__ bool cap_near(float* x, const Cap<Z>& c, bool live) {
  float far[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < TBN; k += 2) {
    float u[2];
    cap_poly(x + k, u, x + k, c);
    far[(k >> 1) & 3] = max3(far[(k >> 1) & 3], u[0], u[1]);
  }
  const bool beyond = live && max3(fmaxf(far[0], far[1]), far[2], far[3]) > c.most;
  return !__any_sync(0xffffffffu, beyond);
}
// The same for any scores, each by its own form (near ones to the same bits: keys that a row
// does not see may send its warp here).  z2: 2 kz log2 e; cl: c log2 e.
template <bool Z>
__device__ __forceinline__ void cap_far(float* x, const Cap<Z>& c, float z2, float cl) {
#pragma unroll
  for (int k = 0; k < TBN; k += 2) {
    float u[2], y[2];
    cap_poly(x + k, u, y, c);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float f = fmaf(-2.f * cl, rcp(1.f + ex2(x[k + e] * z2)), cl);
      x[k + e] = u[e] <= c.most ? y[e] : f;
    }
  }
}
// Scores times `scale`, less the slope times the distance |at - k| of key k.  The
// distance of a tile that lies wholly before or behind the row is linear in k.
__device__ __forceinline__ void bias_scores(float* x, float scale, float slope, float at) {
  if (__all_sync(0xffffffffu, at >= (float)(TBN - 1) || at <= 0.f)) {
    const float ns = at > 0.f ? -slope : slope;
#pragma unroll
    for (int k = 0; k < TBN; k += 2) {
      float y0, y1;
      mul2(y0, y1, x[k], x[k + 1], scale, scale);
      fma2(x[k], x[k + 1], at - (float)k, at - (float)(k + 1), ns, y0, y1);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < TBN; ++k) x[k] = fmaf(-slope, fabsf(at - (float)k), x[k] * scale);
}

// Which of a tile's 128 keys a row sees (bit k of word k / 32): those below its
// limit and, with documents, of its document.  The rows of a warp carry few
// documents as a rule: one ballot per document and word serves all its rows (lane l
// holds the ids of keys l, 32 + l, 64 + l and 96 + l).
__device__ __forceinline__ void seen_keys(uint32_t* seen, int left, bool docs, const int32_t* doc_k,
                                          int t0, int Nk, int docq) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int n = left - 32 * k;
    seen[k] = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
  }
  if (!docs) return;
  int id[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) id[k] = doc_k[min(t0 + 32 * k + lane, Nk - 1)];
  uint32_t todo = __ballot_sync(0xffffffffu, left > 0 && docq >= 0);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  while (todo) {
    const int d = __shfl_sync(0xffffffffu, docq, __ffs(todo) - 1);
    const bool same = docq == d;
    todo &= ~__ballot_sync(0xffffffffu, same);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t on = __ballot_sync(0xffffffffu, id[k] == d);
      if (same) w[k] = on;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) seen[k] &= w[k];
}

__device__ __forceinline__ float max_of(const float* x) {
  float m[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) m[e] = fmaxf(x[e], x[e + 8]);
#pragma unroll
  for (int k = 16; k < TBN; k += 16)
#pragma unroll
    for (int e = 0; e < 8; ++e) m[e] = max3(m[e], x[k + e], x[k + 8 + e]);
  return fmaxf(max3(m[0], m[1], m[2]), max3(max3(m[3], m[4], m[5]), m[6], m[7]));
}

// fp16 probabilities are scaled by 2^7: with the stale maximum they reach 2^15,
// and values down to 2^-21 of the row's largest stay normal numbers.
template <typename T>
constexpr float p_shift() { return sizeof(T) == 2 && std::is_same<T, __half>::value ? 7.f : 0.f; }

// MODE: PLAIN scores, CAP tanh cap, BIAS distance penalty, BOTH of them (or a cap far from the
// scores' size without a penalty).
enum { PLAIN, CAP, BIAS, BOTH };
template <typename T, int D, bool SOLO, int MODE>
__global__ void __launch_bounds__(AM_THREADS, 1)
    k_attend_masked(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AmArgs a) {
  constexpr uint32_t TILE = tile_bytes<D>();
  constexpr int NST = ring<D>(), NBOX = D / 64;
  constexpr bool BIASED = MODE == BIAS || MODE == BOTH, CAPPED = MODE == CAP || MODE == BOTH;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = base;             // two tiles (SOLO: the first)
  uint8_t* sKV = base + 2 * TILE;  // ring: K and V tiles in turn
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + (2 + NST) * TILE);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;
  uint64_t* s_full = bars + 2;   // [2]
  uint64_t* p_full = bars + 4;   // [2] all of P
  uint64_t* p_half = bars + 6;   // [2] P of the tile's first 64 keys
  uint64_t* o_full = bars + 8;   // [2]
  uint64_t* o_free = bars + 10;  // [2]
  uint64_t* drain = bars + 12;
  uint64_t* full = bars + 13;          // [NST]
  uint64_t* empty = bars + 13 + NST;   // [NST]
  uint64_t* it_full = bars + 13 + 2 * NST;          // [ITEMS]
  uint64_t* it_empty = it_full + ITEMS;             // [ITEMS] eight softmax warps, the issuing warp
  Item<SOLO>* ring_items = reinterpret_cast<Item<SOLO>*>(it_empty + ITEMS);
  uint32_t* tmem_base_s = reinterpret_cast<uint32_t*>(ring_items + ITEMS);
  volatile int* abort_s = reinterpret_cast<volatile int*>(tmem_base_s + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::mbar_init(q_full, 1);
    tc::mbar_init(q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(s_full + s, 1);
      tc::mbar_init(p_full + s, TBM);
      tc::mbar_init(p_half + s, TBM);
      tc::mbar_init(o_full + s, 1);
      tc::mbar_init(o_free + s, TBM);
    }
    tc::mbar_init(drain, 1);
    for (int s = 0; s < ITEMS; ++s) {
      tc::mbar_init(it_full + s, 1);
      tc::mbar_init(it_empty + s, 9);
    }
    for (int s = 0; s < NST; ++s) {
      tc::mbar_init(full + s, 1);
      tc::mbar_init(empty + s, 1);
    }
    *abort_s = 0;
    tc::fence_barrier_init();
  }
  if (warp == 9) {
    tc::tmem_alloc(tmem_base_s, TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tbase = *tmem_base_s;
  after_previous();

  // Item k of this block, as a warp of the consumers sees it; false: no more.
  auto next_item = [&](int k, Item<SOLO>& it) {
    const bool got = tc::mbar_wait(it_full + k % ITEMS, (k / ITEMS) & 1, abort_s, WAIT_NS);
    __syncwarp();
    if (!__all_sync(0xffffffffu, got)) return false;
    it = ring_items[k % ITEMS];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(it_empty + k % ITEMS);
    return it.n >= 0;
  };

  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(OTHER_REGS));
  if (warp == 8) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      tc::prefetch_tmap(&tmQ);
      tc::prefetch_tmap(&tmK);
      tc::prefetch_tmap(&tmV);
      int c = 0, items = 0;  // tiles loaded into the ring, items with work
      bool ok = true;
      const uint32_t qbox = a.pack > 1 ? (uint32_t)(a.pack * a.Nq) * 128u : BOX;
      const int rep = a.Hq / a.Hk;
      for (int k = 0; ok; ++k) {
        // blocks take the items forward and backward in turn, or whichever is next
        const int w = a.next_item ? atomicAdd(a.next_item, 1)
                            : k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        Item<SOLO> it;
        if (w < a.n_items)
          it.init(a, w);
        else
          it.n = -1;
        if (k >= ITEMS && !(ok = tc::mbar_wait(it_empty + k % ITEMS, ((k / ITEMS) - 1) & 1, abort_s,
                                               WAIT_NS)))
          break;
        ring_items[k % ITEMS] = it;
        tc::mbar_arrive(it_full + k % ITEMS);
        if (it.n < 0) break;
        if (it.n == 0) continue;
        auto load_kv = [&](const CUtensorMap* m, int t, int mb, int mh) {
          const int s = c % NST;
          if (c >= NST && !tc::mbar_wait(empty + s, ((c / NST) - 1) & 1, abort_s, WAIT_NS))
            return false;
          tc::mbar_expect_tx(full + s, TILE);
          for (int j = 0; j < NBOX; ++j)
            tc::tma_load_4d(sKV + (size_t)s * TILE + j * BOX, m, 64 * j, t * TBN,
                            (it.h0 / rep) * mh, it.b * mb, full + s);
          ++c;
          return true;
        };
        int bits;
        int t = it.entry(0, bits);
        if (!(ok = load_kv(&tmK, t, a.kmul_b, a.kmul_h))) break;
        if (items > 0 && !tc::mbar_wait(q_empty, (items - 1) & 1, abort_s, WAIT_NS)) break;
        const int nq = SOLO ? 1 : 2;
        tc::mbar_expect_tx(q_full, nq * NBOX * qbox);
        for (int s = 0; s < nq; ++s)
          for (int j = 0; j < NBOX; ++j)
            tc::tma_load_4d(sQ + s * TILE + j * BOX, &tmQ, 64 * j, it.q0 + s * TBM,
                            it.h0 * a.qmul_h, it.b * a.qmul_b, q_full);
        ++items;
        for (int i = 0; i < it.n && ok; ++i) {
          if (i > 0) {
            t = it.entry(i, bits);
            if (!(ok = load_kv(&tmK, t, a.kmul_b, a.kmul_h))) break;
          }
          ok = load_kv(&tmV, t, a.vmul_b, a.vmul_h);
        }
      }
      if (*abort_s) {  // let our copies in flight land before the block exits
        for (int k = c - NST; k < c; ++k)
          if (k >= 0) tc::mbar_wait_bounded(full + (k % NST), (k / NST) & 1, 100000000ull);
        if (items > 0) tc::mbar_wait_bounded(q_full, (items - 1) & 1, 100000000ull);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ products
    // All lanes run the loop, one issues: a run of products whose operands come
    // from uniform registers costs the issuing thread less than the tensor core
    // (a lane-0 branch made it the bound: 1,720 cycles to issue a stream's tile
    // of 1,024 cycles of products).
    constexpr bool BF = std::is_same<T, bf16>::value;
    constexpr uint32_t idS = BF ? tc::idesc_bf16(TBM, TBN, 0) : tc::idesc_fp16(TBM, TBN, 0);
    constexpr uint32_t idPV = BF ? tc::idesc_bf16(TBM, D, 1) : tc::idesc_fp16(TBM, D, 1);
    const uint64_t qd = tc::smem_desc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t kd = tc::smem_desc_sw128(smem_u32(sKV), 16, 1024);
    const uint64_t vd = tc::smem_desc_sw128(smem_u32(sKV), BOX, 1024);
    int c = 0;                           // ring entries of the items before this one
    int np[2] = {0, 0}, no[2] = {0, 0};  // P tiles consumed, items finished, per stream
    int items = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool got = tc::mbar_wait(bar, parity, abort_s, WAIT_NS);
      return __all_sync(0xffffffffu, got) != 0;
    };
    auto wait_ring = [&](int k) { return wait(full + k % NST, (k / NST) & 1); };
    auto commit = [&](uint64_t* bar) {
      if (tc::elect_one()) tc::mma_commit(bar);
      __syncwarp();
    };
    auto issue_s = [&](int s, int k) {
      tc::tc_fence_after();
      const uint64_t q = qd + (SOLO ? 0 : (uint64_t)(s * (TILE >> 4)));
      const uint64_t b = kd + (uint64_t)((k % NST) * (TILE >> 4));
      if (tc::elect_one()) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * BOX + (ks & 3) * 32) >> 4;
          tc::mma_ss(tbase + s * 128, q + off, b + off, idS, ks > 0);
        }
        tc::mma_commit(s_full + s);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int s, int k, auto half, uint32_t accumulate) {
      tc::tc_fence_after();
      const uint64_t b = vd + (uint64_t)((k % NST) * (TILE >> 4));
      constexpr int K0 = decltype(half)::value * (TBN / 32);
      if (tc::elect_one()) {
#pragma unroll
        for (int kk = K0; kk < K0 + TBN / 32; ++kk)
          tc::mma_ts(tbase + O_COL + s * 128, tbase + s * 128 + kk * 8, b + kk * (2048 >> 4), idPV,
                     kk == 0 ? accumulate : 1u);
      }
      __syncwarp();
    };
    bool ok = true;
    for (int k = 0; ok; ++k) {
      Item<SOLO> it;
      if (!next_item(k, it)) break;
      if (it.n == 0) continue;
      if (!(ok = wait(q_full, items & 1))) break;
      bool first[2] = {true, true}, done[2] = {false, false};
      // the first tile's scores (SOLO: of both streams' first tiles)
      if (!(ok = wait_ring(c))) break;
      uint32_t on = it.streams(0), on_next;  // the streams that visit tile i and tile i + AHEAD
      if (SOLO || (on & 1)) issue_s(0, c);
      if (!SOLO && (on & 2)) issue_s(1, c);
      commit(empty + c % NST);
      if (SOLO && it.n > 1) {
        if (!(ok = wait_ring(c + 2))) break;
        issue_s(1, c + 2);
        commit(empty + (c + 2) % NST);
      }
      constexpr int AHEAD = SOLO ? 2 : 1;  // tiles between a stream's product and its next scores
      if (it.n <= AHEAD) commit(q_empty);
      for (int i = 0; i < it.n; ++i, on = on_next) {
        const int kv = c + 2 * i + 1, kn = c + 2 * (i + AHEAD);
        const bool more = i + AHEAD < it.n;
        if (SOLO) on = 1u << (i & 1);
        on_next = SOLO ? on : more ? it.streams(i + AHEAD) : 0u;
        if (!(ok = wait_ring(kv))) break;
        bool have_k = false;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (on >> s & 1) {
            if (!(ok = wait(p_half + s, np[s] & 1))) break;
            if (first[s] && no[s] > 0 && !(ok = wait(o_free + s, (no[s] - 1) & 1))) break;
            issue_pv(s, kv, std::integral_constant<int, 0>{}, !first[s]);
            if (!(ok = wait(p_full + s, np[s] & 1))) break;
            issue_pv(s, kv, std::integral_constant<int, 1>{}, 1u);
            ++np[s];
            first[s] = false;
            if (!SOLO && i == it.last[s]) {
              commit(o_full + s);
              done[s] = true;
            }
          }
          if (more && (on_next >> s & 1)) {
            if (!have_k && !(ok = wait_ring(kn))) break;
            have_k = true;
            issue_s(s, kn);
          }
        }
        if (!ok) break;
        commit(empty + kv % NST);
        if (more) {
          if (!have_k && !(ok = wait_ring(kn))) break;
          commit(empty + kn % NST);
          if (i + AHEAD + 1 == it.n) commit(q_empty);
        }
      }
      if (!ok) break;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (!first[s]) {
          if (SOLO || !done[s]) commit(o_full + s);
          ++no[s];
        }
      c += 2 * it.n;
      ++items;
    }
    commit(drain);
    tc::mbar_wait_bounded(drain, 0, WAIT_NS);
  }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(SOFTMAX_REGS));
    const int s = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_f = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t scol = tbase + lane_f + s * 128, ocol = tbase + lane_f + O_COL + s * 128;
    const float scale_log2 = a.scale * LOG2E;
    Cap<MODE == BOTH> cap;
    if (CAPPED) cap.init(a.scale, a.softcap, a.kz);
    int np = 0, no = 0, c = 0;  // tiles and items this stream has had, ring entries so far
    bool ok = true;
    for (int k = 0; ok; ++k) {
      Item<SOLO> it;
      if (!next_item(k, it)) break;
      // this thread's row: query head and query
      int h = it.h0, qi = it.q0 + (SOLO ? 0 : s * TBM) + row;
      bool live = qi < a.Nq;
      if (a.pack > 1) {
        const int g = row / a.Nq, rep = a.Hq / a.Hk;
        qi = row - g * a.Nq;
        h = it.h0 + g;
        live = g < a.pack && h < (it.h0 / rep + 1) * rep && (SOLO || s == 0);
        if (!live) qi = 0, h = it.h0;
      }
      const int whole = it.lim.limit(it.q0 + (SOLO ? 0 : s * TBM));  // keys every row of the tile sees
      const int lim = live ? it.lim.limit(qi) : 0;
      const int docq = a.doc_q && live ? a.doc_q[(int64_t)it.b * a.Nq + qi] : 0;
      const float slope = BIASED && a.slopes ? a.slopes[h] * LOG2E : 0.f;
      const int32_t* dk = a.doc_k ? a.doc_k + (int64_t)it.b * a.Nk : nullptr;
      const bool work = __any_sync(0xffffffffu, live);  // a warp without rows only keeps step
      const int place = BIASED ? it.lim.nearest(qi) : 0;
      float m = -INFINITY, l = 0.f;
      bool first = true;
      int far = 0;
      for (int i = 0; i < it.n; ++i) {
        int bits;
        const int t = it.entry(i, bits);
        if (SOLO ? (i & 1) != s : !(bits >> s & 1)) continue;
        const int t0 = t * TBN;
        const bool doc_part = dk && !(bits >> (SOLO ? 2 : 2 + s) & 1);
        const bool part = doc_part || t0 + TBN > whole;  // keys of the tile are hidden from rows
        uint32_t seen[4];
        if (part && work) seen_keys(seen, lim - t0, doc_part, dk, t0, a.Nk, docq);
        const bool got_s = tc::mbar_wait(s_full + s, np & 1, abort_s, WAIT_NS);
        __syncwarp();
        if (!__all_sync(0xffffffffu, got_s)) {
          ok = false;
          break;
        }
        ++np;
        tc::tc_fence_after();
        float x[TBN];
        auto load = [&]() {
          uint32_t* sr = reinterpret_cast<uint32_t*>(x);
#pragma unroll
          for (int k = 0; k < 4; ++k) tc::tmem_ld32(scol + 32 * k, sr + 32 * k);
          tc::tmem_wait_ld();
        };
        auto hide = [&](float value) {  // the scores of the keys that the row does not see
#pragma unroll
          for (int k = 0; k < TBN; ++k)
            if (!(seen[k / 32] & (1u << (k % 32)))) x[k] = value;
        };
        auto take = [&]() {  // the row's scores, transformed and masked
          load();
          if (CAPPED && !far && !cap_near(x, cap, live)) {
            far = 1;  // for the rest of the item: such scores seldom come alone
            load();
          }
          // The compiler must not see that `far` follows from the branch above: it then makes one
          // block of the loads and the far form, whose spills the near form pays for (2 x 16 heads
          // x 4,097, d = 64, cap and prefix 270 -> 282 us; 24 heads x 8,192, cap and slopes 1,316 ->
          // 1,760).
          if (CAPPED) asm volatile("" : "+r"(far));
          if (CAPPED && far) cap_far(x, cap, 2.f * LOG2E * a.kz, a.softcap * LOG2E);
          if (BIASED && a.slopes)  // (BIAS always: the branch keeps the loads from spilling)
            bias_scores(x, MODE == BIAS ? scale_log2 : 1.f, slope, (float)(place - t0));
          if (part) hide(-INFINITY);
        };
        const float sl2 = MODE == PLAIN ? scale_log2 : 1.f;
        uint32_t pr[32];
        float sum4[4];
        // P of 64 keys from key K0 on, rounded to the 16-bit type: the product takes both operands
        // in one type.  That is half a step a probability, at random: O's error against 64 bits is
        // 0.0019 of its size instead of the 0.0017 of its own rounding where few keys count (slopes),
        // less where many do.  The sum takes them unrounded.  A row that has seen nothing keeps m = -inf;
        // what it adds up meanwhile is dropped with the first score it sees, or at the end.
        auto exps = [&](auto from) {
          constexpr int K0 = decltype(from)::value;
          const float neg = m == -INFINITY ? 0.f : p_shift<T>() - m;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float x0, x1;
            fma2(x0, x1, x[K0 + 2 * e], x[K0 + 2 * e + 1], sl2, neg);
            const float p0 = ex2(x0), p1 = ex2(x1);
            add2(sum4[2 * (e & 1)], sum4[2 * (e & 1) + 1], p0, p1);
            pr[e] = pack2<T>(p0, p1);
          }
        };
        using Lo = std::integral_constant<int, 0>;
        using Hi = std::integral_constant<int, TBN / 2>;
        // A row's maximum is moved only when it grew by more than 2^8: then what was
        // added up so far is scaled down.
        auto move_max = [&](bool grown, float mx) {
          const float top = grown ? mx : m;
          if (!first) {  // the products before S(i) are done: O is at rest
            const float corr = grown ? ex2(m - top) : 1.f;
            l *= corr;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              uint32_t o[16];
              __syncwarp();
              tc::tmem_ld16(ocol + 16 * k, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              __syncwarp();
              tc::tmem_st16(ocol + 16 * k, o);
            }
          }
          m = top;
        };
        // BIAS, BOTH: where every probability of the warp's rows would be flushed to 0 (a
        // distance penalty far from the rows), there is no exponential to take.
        bool nothing = false;
        if (BIASED) {
          if (work) {
            take();
            const float mx = max_of(x);
            const bool grown = live && mx > m + 8.f;
            if (__any_sync(0xffffffffu, grown)) move_max(grown, mx);
            nothing = __all_sync(0xffffffffu, !live || mx < m - 140.f);
            sum4[0] = sum4[1] = sum4[2] = sum4[3] = 0.f;
            if (nothing) {
#pragma unroll
              for (int e = 0; e < 32; ++e) pr[e] = 0u;
            } else {
              exps(Lo{});
            }
          }
        } else {
          // the first half's exponentials go ahead with the maximum so far, under
          // the search for the new one; they are seldom taken again (the first
          // tile's wait for its maximum)
          while (work) {
            take();
            const float mx = max_of(x) * sl2;
            if (first) m = mx;
            sum4[0] = sum4[1] = sum4[2] = sum4[3] = 0.f;
            exps(Lo{});
            const bool grown = live && mx > m + 8.f;
            if (!__any_sync(0xffffffffu, grown)) break;
            move_max(grown, mx);
          }
        }
        first = false;
        bool got_v = true;
        if (bits & 16) {  // zero the V rows of keys that count for nobody
          const int kv = c + 2 * i + 1;
          got_v = tc::mbar_wait(full + kv % NST, (kv / NST) & 1, abort_s, WAIT_NS);
          const int j = t0 + row;
          if (got_v && (j >= it.lim.end || (dk && dk[j] < 0))) {
            uint8_t* v = sKV + (size_t)(kv % NST) * TILE + row * 128;
#pragma unroll
            for (int k = 0; k < NBOX; ++k)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint4*>(v + k * BOX + 16 * e) = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (!__all_sync(0xffffffffu, got_v)) {
            ok = false;
            break;
          }
        }
        if (work) {
          __syncwarp();
          tc::tmem_st32(scol, pr);
          tc::tmem_wait_st();
        }
        tc::tc_fence_before();
        tc::mbar_arrive(p_half + s);
        if (work) {
          if (!nothing) exps(Hi{});
          __syncwarp();
          tc::tmem_st32(scol + 32, pr);
          l += (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
          tc::tmem_wait_st();
        }
        tc::tc_fence_before();
        tc::mbar_arrive(p_full + s);
      }
      if (!ok) break;
      c += 2 * it.n;
      const bool any = !first;
      if (m == -INFINITY && l == l) l = 0.f;  // the row saw no key
      if (any) {
        const bool got_o = tc::mbar_wait(o_full + s, no & 1, abort_s, WAIT_NS);
        __syncwarp();
        if (!__all_sync(0xffffffffu, got_o)) {
          ok = false;
          break;
        }
        ++no;
        tc::tc_fence_after();
      }
      if (it.part >= 0) {
        const int64_t part = (it.part + s) * a.part_rows + row;
        if (live) {
          a.part_ml[2 * part] = m;
          a.part_ml[2 * part + 1] = l;
        }
        if (any)
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            uint32_t o[32];
            __syncwarp();
            tc::tmem_ld32(ocol + 32 * k, o);
            tc::tmem_wait_ld();
            if (live) {
              uint4* d = reinterpret_cast<uint4*>(a.part_o + part * D + 32 * k);
#pragma unroll
              for (int e = 0; e < 4; ++e) store32(d + 2 * e, o + 8 * e);
            }
          }
      } else {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        // NaN sums stay NaN
        const float f = l == l ? inv : l;
        uint4* d = reinterpret_cast<uint4*>(static_cast<T*>(a.O) + it.b * a.os[0] + h * a.os[1] +
                                            (int64_t)qi * a.os[2]);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t o[32];
          if (any) {
            __syncwarp();
            tc::tmem_ld32(ocol + 32 * k, o);
            tc::tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (live) {
            uint32_t u[16];
#pragma unroll
            for (int g = 0; g < 16; ++g)
              u[g] = l == 0.f ? 0u
                              : pack2<T>(__uint_as_float(o[2 * g]) * f,
                                         __uint_as_float(o[2 * g + 1]) * f);
            if (a.o_wide) {
              store32(d + 4 * k, u);
              store32(d + 4 * k + 2, u + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                d[4 * k + e] = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
            }
          }
        }
        if (live && a.lse) {
          float lse = l == 0.f ? -INFINITY : (m - p_shift<T>()) * LN2 + logf(l);
          if (BIASED && a.slopes && l != 0.f) lse = fmaf(-a.slopes[h], it.lim.beyond(qi), lse);
          a.lse[((int64_t)it.b * a.Hq + h) * a.Nq + qi] = lse;
        }
      }
      if (any) {
        tc::tc_fence_before();
        tc::mbar_arrive(o_free + s);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (threadIdx.x == 0 && *abort_s) report_timeout(a.status, a.words);
  if (warp == 9) {
    __syncwarp();
    tc::tmem_dealloc(tbase, TMEM_COLS);
  }
}

// Add up the partial results of the rows of the split tiles: WARPS warps to a
// row, each with every WARPS-th of the row's parts (2 nsplit of them in the SOLO
// form, nsplit in the other), in an order that is fixed.
template <typename T, int D, bool SOLO, int WARPS>
__global__ void __launch_bounds__(128) k_am_join(const __grid_constant__ AmArgs a) {
  constexpr int ROWS = 4 / WARPS, E = D / 32;
  __shared__ float sm[4], sl[4], so[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  after_previous();
  const int per_tile = SOLO ? a.part_rows : 2 * TBM;
  const int64_t at = (int64_t)blockIdx.x * ROWS + warp / WARPS;
  const int tt = (int)(at / per_tile), r = (int)(at % per_tile);  // split tile, its row
  if (tt >= a.n_tiles - a.n_whole) return;
  Item<SOLO> it;
  it.place(a, a.n_whole + tt);
  const int s = SOLO ? 0 : r / TBM, row = SOLO ? r : r % TBM, b = it.b;
  int h = it.h0, qi = it.q0 + r;
  if (a.pack > 1) {  // (SOLO)
    const int rep = a.Hq / a.Hk;
    h += row / a.Nq;
    qi = row % a.Nq;
    if (h >= (it.h0 / rep + 1) * rep) return;
  }
  if (qi >= a.Nq) return;
  const int np = SOLO ? 2 * a.nsplit : a.nsplit, step = SOLO ? 1 : 2;
  const int64_t p0 = ((int64_t)tt * a.nsplit * 2 + s) * a.part_rows + row;
  const int64_t pstep = (int64_t)step * a.part_rows;
  const int first = warp % WARPS;
  float M = -INFINITY;
  for (int p = first + WARPS * lane; p < np; p += WARPS * 32)
    M = fmaxf(M, a.part_ml[2 * (p0 + p * pstep)]);
  M = warp_max(M);
  float o[E] = {}, l = 0.f;
#pragma unroll 4
  for (int p = first; p < np; p += WARPS) {
    const int64_t i = p0 + p * pstep;
    const float m = a.part_ml[2 * i], lp = a.part_ml[2 * i + 1];
    if (lp == 0.f) continue;  // saw nothing; its O is not written
    const float w = ex2(m - M);
    l += w * lp;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(w, a.part_o[i * D + E * lane + e], o[e]);
  }
  if (WARPS > 1) {
    if (lane == 0) sm[warp] = M, sl[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][E * lane + e] = o[e];
    __syncthreads();
    if (first) return;
    float top = M;
    for (int i = 1; i < WARPS; ++i) top = fmaxf(top, sm[warp + i]);
    float w = M == -INFINITY ? 0.f : ex2(M - top);
    l *= w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= w;
    for (int i = 1; i < WARPS; ++i) {
      if (sm[warp + i] == -INFINITY && sl[warp + i] == 0.f) continue;
      w = ex2(sm[warp + i] - top);
      l = fmaf(w, sl[warp + i], l);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(w, so[warp + i][E * lane + e], o[e]);
    }
    M = top;
  }
  const float f = l != 0.f ? 1.f / l : 0.f;
  T* O = static_cast<T*>(a.O) + b * a.os[0] + h * a.os[1] + (int64_t)qi * a.os[2] + E * lane;
  const uint32_t u0 = pack2<T>(o[0] * f, o[1] * f);
  if (E == 4) {
    *reinterpret_cast<uint2*>(O) = make_uint2(u0, pack2<T>(o[E - 2] * f, o[E - 1] * f));
  } else {
    *reinterpret_cast<uint32_t*>(O) = u0;
  }
  if (a.lse && lane == 0) {
    float lse = l == 0.f ? -INFINITY : (M - p_shift<T>()) * LN2 + logf(l);
    if (a.slopes && l != 0.f) {
      it.lim.init(a, b);
      lse = fmaf(-a.slopes[h], it.lim.beyond(qi), lse);
    }
    a.lse[((int64_t)b * a.Hq + h) * a.Nq + qi] = lse;
  }
}

// The key tiles that a row tile has to visit under documents: a block per (row
// tile, batch), a warp per key tile, 32 tiles at a time.  A tile whose ids do
// not meet the rows' range is left out; it is whole for a stream when rows and
// keys all carry one id.
template <bool SOLO>
__global__ void __launch_bounds__(1024) k_am_documents(const __grid_constant__ AmArgs a,
                                                       int32_t* count, int32_t* list) {
  __shared__ int lo[2], hi[2], neg[2], final_entry[2], entry[32];
  const int b = blockIdx.y, blk = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int span = SOLO ? TBM : 2 * TBM, q0 = blk * span;
  after_previous();
  if (threadIdx.x < 2) {
    lo[threadIdx.x] = INT32_MAX;
    hi[threadIdx.x] = -1;
    neg[threadIdx.x] = 0;
    final_entry[threadIdx.x] = -1;
  }
  __syncthreads();
  if ((int)threadIdx.x < span && q0 + (int)threadIdx.x < a.Nq) {
    const int id = a.doc_q[(int64_t)b * a.Nq + q0 + threadIdx.x], s = threadIdx.x / TBM;
    if (id >= 0) {
      atomicMin(&lo[s], id);
      atomicMax(&hi[s], id);
    } else {
      neg[s] = 1;
    }
  }
  __syncthreads();
  Limits lim;
  lim.init(a, b);
  int nt[2];
  for (int s = 0; s < 2; ++s) {
    const int first = SOLO ? q0 : q0 + s * TBM, last = min(first + TBM, a.Nq) - 1;
    nt[s] = first < a.Nq ? (lim.limit(last) + TBN - 1) / TBN : 0;
  }
  const int64_t at = (int64_t)b * a.nqb + blk;
  int32_t* out = list + at * a.ktiles;
  int n = 0;
  const int most = max(nt[0], nt[1]);
  for (int tb = 0; tb < most; tb += 32) {
    const int t = tb + warp;
    int bits = 0;
    if (t < most) {
      int kl = INT32_MAX, kh = -1;
      bool dead = (t + 1) * TBN > lim.end;
      for (int k = 0; k < 4; ++k) {
        const int j = t * TBN + 32 * k + lane;
        const int id = j < lim.end ? a.doc_k[(int64_t)b * a.Nk + j] : -1;
        if (id >= 0) {
          kl = min(kl, id);
          kh = max(kh, id);
        } else {
          dead = true;
        }
      }
      kl = __reduce_min_sync(0xffffffffu, kl);
      kh = __reduce_max_sync(0xffffffffu, kh);
      dead = __any_sync(0xffffffffu, dead);
      for (int s = 0; s < 2; ++s) {
        const int r = SOLO ? 0 : s;
        if (t < nt[r] && kl <= hi[r] && lo[r] <= kh) {
          bits |= 1 << s;
          if (kl == kh && lo[r] == hi[r] && !neg[r] && !dead) bits |= 4 << s;
        }
      }
      if (dead) bits |= 16;
    }
    if (lane == 0) entry[warp] = bits & 3 ? t << 5 | bits : -1;
    __syncthreads();
    if (warp == 0) {
      const int e = entry[lane];
      const uint32_t keep = __ballot_sync(0xffffffffu, e >= 0);
      if (e >= 0) {
        const int slot = n + __popc(keep & ((1u << lane) - 1));
        out[slot] = e;
        if (e & 1) atomicMax(&final_entry[0], slot);
        if (e & 2) atomicMax(&final_entry[1], slot);
      }
      n += __popc(keep);
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    count[4 * at] = n;
    count[4 * at + 1] = final_entry[0];
    count[4 * at + 2] = final_entry[1];
    if (at == 0 && a.next_item) *a.next_item = 0;
  }
}

// The plan of a call: which form, how many items, what the workspace holds.
struct Plan {
  bool solo;
  int pack, ntile_h, nqb, nsplit, n_items, ktiles, part_rows, by_block, n_tiles, n_whole;
  size_t words_off, next_off, count_off, list_off, o_off, ml_off, total;
};

Plan make_plan(const spr_masked_params& p, int sms) {
  Plan q{};
  const int rep = p.Hq / p.Hk;
  // Up to 128 rows that share their keys form one tile: the query tokens of a
  // head, or of as many heads of the key head as fit.
  q.solo = p.Nq <= TBM;
  q.pack = q.solo && 2 * p.Nq <= TBM ? (rep < TBM / p.Nq ? rep : TBM / p.Nq) : 1;
  q.ktiles = (p.Nk + TBN - 1) / TBN;
  // ... which over up to three key tiles one stream of the other form takes, one
  // after the other: a tile is 1.4 us, the join it saves 3.
  if (q.ktiles <= 3) q.solo = false;
  q.ntile_h = p.Hk * ((rep + q.pack - 1) / q.pack);
  q.nqb = q.solo ? 1 : (p.Nq + 2 * TBM - 1) / (2 * TBM);
  const int64_t tiles = (int64_t)p.B * q.ntile_h * q.nqb;
  // Key splits with the least estimated time, in cycles of an SM: a key tile
  // takes a SOLO block what its 4 d 128 bytes take at 24 bytes a cycle (the
  // SM's share of HBM), the other form about 3,300 cycles of softmax for its two
  // streams; an item costs 2,000 or 4,000 cycles to start and end; the join a launch and
  // the partial results' way out and back.  At least two tiles to a split.
  const double step = q.solo ? 4.0 * p.d * TBN / 24 : 3300.0;
  const double part = q.solo ? 2.0 * q.pack * p.Nq * p.d * 4 : 2.0 * TBM * p.d * 4;
  const int most = q.ktiles / 2 < 1 ? 1 : q.ktiles / 2;
  double best = 0;
  for (int n = 1; n <= most && (n == 1 || tiles * n <= (q.solo ? 16 : 1) * (int64_t)sms); ++n) {
    const int64_t rounds = (tiles * n + sms - 1) / sms;
    const bool joined = q.solo || n > 1;
    const double cost = (double)rounds * ((q.ktiles + n - 1) / n * step + (q.solo ? 2000.0 : 4000.0)) +
                        (joined ? 6000.0 + 30.0 * n + 2.0 * tiles * n * part / 3500.0 : 0.0);
    if (n == 1 || cost < best) {
      best = cost;
      q.nsplit = n;
    }
  }
  // Causal items differ in length: heaviest first over all heads, as long as
  // the keys and values of all heads stay in L2 together.
  q.by_block = p.causal && !q.solo && 4.0 * p.B * p.Hk * p.Nk * p.d <= 48e6;
  q.n_tiles = (int)tiles;
  q.n_whole = q.solo || q.nsplit > 1 ? 0 : q.n_tiles;
  // More tiles than SMs, of one length: those of a last round that leaves half
  // of the SMs idle or more are split over them (24 heads x 8,192 x 8,192, 768 tiles on
  // 148 SMs: 951 -> 854 us).
  const int left = q.n_tiles % sms;
  if (!p.causal && q.n_whole > sms && left && sms / left >= 2 && q.ktiles >= 4) {
    const int n = sms / left < q.ktiles / 2 ? sms / left : q.ktiles / 2;
    if (q.ktiles * step * (n - 1) / n > 25000.0) {
      q.nsplit = n;
      q.n_whole = q.n_tiles - left;
    }
  }
  const int split_items = (q.n_tiles - q.n_whole) * q.nsplit;
  q.n_items = q.n_whole + split_items;
  q.part_rows = q.solo ? q.pack * p.Nq : TBM;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t off = at;
    at += (bytes + 255) / 256 * 256;
    return off;
  };
  q.words_off = take(16);
  q.next_off = take(4);
  q.count_off = take((size_t)p.B * q.nqb * 16);
  q.list_off = take((size_t)p.B * q.nqb * q.ktiles * 4);
  q.o_off = take((size_t)split_items * 2 * q.part_rows * p.d * 4);
  q.ml_off = take((size_t)split_items * 2 * q.part_rows * 8);
  q.total = at;
  return q;
}

// [B, H, N, d] as a TMA map of boxes of `rows` x `heads` rows of 64 channels.
// A dimension of stride 0 becomes one entry whose coordinate stays 0.
bool make_map(CUtensorMap* m, const void* ptr, CUtensorMapDataType dt, int B, int H, int N, int d,
              const int64_t* s, int rows, int heads, int* mul_b, int* mul_h) {
  *mul_b = B > 1 && s[0] ? 1 : 0;
  *mul_h = H > 1 && s[1] ? 1 : 0;
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)N, (uint64_t)(*mul_h ? H : 1),
                            (uint64_t)(*mul_b ? B : 1)};
  auto bytes = [&](int64_t st, bool on) { return on && st ? (uint64_t)st * 2 : (uint64_t)d * 2; };
  const uint64_t strides[3] = {bytes(s[2], N > 1), bytes(s[1], *mul_h), bytes(s[0], *mul_b)};
  for (uint64_t st : strides)
    if (st >> 40) return false;
  const uint32_t box[4] = {64, (uint32_t)rows, (uint32_t)heads, 1};
  return encode_tmap(m, dt, 4, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename T, int D, bool SOLO, int MODE>
cudaError_t launch(const AmArgs& a, const CUtensorMap& q, const CUtensorMap& k,
                   const CUtensorMap& v, int sms, cudaStream_t st) {
  auto kern = k_attend_masked<T, D, SOLO, MODE>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kern, smem_bytes<D>(), done);
  if (e != cudaSuccess) return e;
  spr_launch_early(kern, a.n_items < sms ? a.n_items : sms, AM_THREADS, smem_bytes<D>(), st, q, k, v, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.n_whole < a.n_tiles) {
    const int64_t rows = (int64_t)(a.n_tiles - a.n_whole) * (SOLO ? a.part_rows : 2 * TBM);
    // a warp goes through four parts in about 1 us; few rows with many parts get four warps each
    if ((SOLO ? 2 : 1) * a.nsplit > 8 && rows <= 65536)
      spr_launch_early(k_am_join<T, D, SOLO, 4>, (unsigned)rows, 128, 0, st, a);
    else
      spr_launch_early(k_am_join<T, D, SOLO, 1>, (unsigned)((rows + 3) / 4), 128, 0, st, a);
    e = cudaGetLastError();
  }
  return e;
}

template <typename T, int D>
cudaError_t launch_for(bool solo, const AmArgs& a, const CUtensorMap& q, const CUtensorMap& k,
                       const CUtensorMap& v, int sms, cudaStream_t st) {
  if (a.softcap > 0.f && (a.slopes || !cap_is_usual(a.scale, a.softcap)))
    return solo ? launch<T, D, true, BOTH>(a, q, k, v, sms, st)
                : launch<T, D, false, BOTH>(a, q, k, v, sms, st);
  if (a.slopes)
    return solo ? launch<T, D, true, BIAS>(a, q, k, v, sms, st)
                : launch<T, D, false, BIAS>(a, q, k, v, sms, st);
  if (a.softcap > 0.f)
    return solo ? launch<T, D, true, CAP>(a, q, k, v, sms, st)
                : launch<T, D, false, CAP>(a, q, k, v, sms, st);
  return solo ? launch<T, D, true, PLAIN>(a, q, k, v, sms, st)
              : launch<T, D, false, PLAIN>(a, q, k, v, sms, st);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool strides_fit(const int64_t* s, int B, int H, int N, bool out) {
  const int size[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    if (s[i] < 0 || (size[i] > 1 && s[i] % 8)) return false;
    if (size[i] > 1 && s[i] == 0 && (out || i == 2)) return false;
  }
  return true;
}

spr_status check(const spr_masked_params* p) {
  if (!p) return SPR_EINVAL;
  if (p->B < 1 || p->Hq < 1 || p->Hk < 1 || p->Nq < 1 || p->Nk < 1 || p->Hq % p->Hk)
    return SPR_EINVAL;
  if (p->d != 64 && p->d != 128) return SPR_EUNSUPPORTED;
  if (p->dtype != SPR_BF16 && p->dtype != SPR_FP16) return SPR_EINVAL;
  if (!isfinite(p->scale) || !isfinite(p->softcap) || p->softcap < 0.f) return SPR_EINVAL;
  if (p->causal != 0 && p->causal != 1) return SPR_EINVAL;
  if (p->q_start != SPR_ALIGN_END && (p->q_start < -(1 << 30) || p->q_start > (1 << 30)))
    return SPR_EINVAL;
  if (p->Nq > (1 << 30) || p->Nk > (1 << 30) || p->B > 65535 || p->Hq > 65535 ||
      (int64_t)p->B * p->Hq * p->Nq > (1 << 30))
    return SPR_EUNSUPPORTED;
  // (Q's too: packed heads are one box of its tensor map)
  if (!strides_fit(p->q_strides, p->B, p->Hq, p->Nq, true) ||
      !strides_fit(p->k_strides, p->B, p->Hk, p->Nk, false) ||
      !strides_fit(p->v_strides, p->B, p->Hk, p->Nk, false) ||
      !strides_fit(p->o_strides, p->B, p->Hq, p->Nq, true))
    return SPR_EUNSUPPORTED;
  return SPR_OK;
}

}  // namespace
}  // namespace spr

using namespace spr;

extern "C" size_t sparsepr_attend_masked_workspace(const spr_masked_params* p) {
  return check(p) == SPR_OK ? make_plan(*p, num_sms()).total : 0;
}

extern "C" spr_status sparsepr_attend_masked(const spr_masked_params* p, const void* Q,
                                             const void* K, const void* V, const int32_t* k_len,
                                             const int32_t* doc_q, const int32_t* doc_k,
                                             const int32_t* prefix, const float* slopes, void* O,
                                             float* lse, void* ws, size_t ws_bytes,
                                             int32_t* status, void* stream) {
  const spr_status s = check(p);
  if (s != SPR_OK) return s;
  if (!Q || !K || !V || !O || (!doc_q != !doc_k) || (prefix && !p->causal)) return SPR_EINVAL;
  if (!ws || !aligned(ws, 256) || ws_bytes < sparsepr_attend_masked_workspace(p))
    return SPR_EWORKSPACE;
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(O, 16) ||
      !aligned(lse, 4) || !aligned(k_len, 4) || !aligned(doc_q, 4) || !aligned(doc_k, 4) ||
      !aligned(prefix, 4) || !aligned(slopes, 4) || !aligned(status, 4))
    return SPR_EUNSUPPORTED;
  const int sms = num_sms();
  const Plan q = make_plan(*p, sms);
  AmArgs a{};
  a.O = O;
  a.lse = lse;
  a.k_len = k_len;
  a.doc_q = doc_q;
  a.doc_k = doc_k;
  a.prefix = prefix;
  a.slopes = slopes;
  for (int i = 0; i < 3; ++i) a.os[i] = p->o_strides[i];
  a.o_wide = aligned(O, 32) && (a.os[0] | a.os[1] | a.os[2]) % 16 == 0;
  a.B = p->B;
  a.Hq = p->Hq;
  a.Hk = p->Hk;
  a.Nq = p->Nq;
  a.Nk = p->Nk;
  a.causal = p->causal;
  a.q_start = p->q_start;
  a.scale = p->scale > 0.f ? p->scale : 1.f / sqrtf((float)p->d);
  // A cap 2^60 times past what a score of 1 becomes leaves all scores as they are in fp32.
  a.softcap = p->softcap > 0x1p60f * a.scale ? 0.f : p->softcap;
  a.kz = fminf(a.scale / a.softcap, FLT_MAX);  // a score of 0 stays one under the smallest caps
  a.pack = q.pack;
  a.ntile_h = q.ntile_h;
  a.nqb = q.nqb;
  a.nsplit = q.nsplit;
  a.by_block = q.by_block;
  a.n_items = q.n_items;
  a.n_tiles = q.n_tiles;
  a.n_whole = q.n_whole;
  if (q.n_whole && (doc_q || k_len)) {  // tiles of different lengths: none is split
    a.nsplit = 1;
    a.n_items = a.n_whole = q.n_tiles;
  }
  uint8_t* base = static_cast<uint8_t*>(ws);
  int32_t* count = reinterpret_cast<int32_t*>(base + q.count_off);
  int32_t* list = reinterpret_cast<int32_t*>(base + q.list_off);
  a.doc_count = count;
  // Items of very different length are taken as blocks come free: documents, and
  // lengths where each block has several items (the counter costs a memset).
  const bool uneven = doc_q || (k_len && p->B > 1 && a.n_items > 2 * sms);
  a.next_item = uneven && a.n_items > sms ? reinterpret_cast<int*>(base + q.next_off) : nullptr;
  a.doc_list = list;
  a.ktiles = q.ktiles;
  a.part_o = reinterpret_cast<float*>(base + q.o_off);
  a.part_ml = reinterpret_cast<float*>(base + q.ml_off);
  a.part_rows = q.part_rows;
  a.status = status;
  a.words = reinterpret_cast<int32_t*>(base + q.words_off);
  const CUtensorMapDataType dt = p->dtype == SPR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap mq, mk, mv;
  if (!tmap_available()) return SPR_ECUDA;
  if (!make_map(&mq, Q, dt, p->B, p->Hq, p->Nq, p->d, p->q_strides, q.pack > 1 ? p->Nq : TBM,
                q.pack, &a.qmul_b, &a.qmul_h) ||
      !make_map(&mk, K, dt, p->B, p->Hk, p->Nk, p->d, p->k_strides, TBN, 1, &a.kmul_b, &a.kmul_h) ||
      !make_map(&mv, V, dt, p->B, p->Hk, p->Nk, p->d, p->v_strides, TBN, 1, &a.vmul_b, &a.vmul_h))
    return SPR_EUNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (status && cudaMemsetAsync(status, 0, 4 * sizeof(int32_t), st) != cudaSuccess)
    return SPR_ECUDA;
  if (a.next_item && !doc_q && cudaMemsetAsync(a.next_item, 0, 4, st) != cudaSuccess)
    return SPR_ECUDA;
  if (doc_q) {
    const dim3 grid(q.nqb, p->B);
    if (q.solo)
      spr_launch_early(k_am_documents<true>, grid, 1024, 0, st, a, count, list);
    else
      spr_launch_early(k_am_documents<false>, grid, 1024, 0, st, a, count, list);
    if (cudaGetLastError() != cudaSuccess) return SPR_ECUDA;
  }
  cudaError_t e;
  if (p->dtype == SPR_BF16)
    e = p->d == 64 ? launch_for<bf16, 64>(q.solo, a, mq, mk, mv, sms, st)
                   : launch_for<bf16, 128>(q.solo, a, mq, mk, mv, sms, st);
  else
    e = p->d == 64 ? launch_for<__half, 64>(q.solo, a, mq, mk, mv, sms, st)
                   : launch_for<__half, 128>(q.solo, a, mq, mk, mv, sms, st);
  return e == cudaSuccess ? SPR_OK : SPR_ECUDA;
}
