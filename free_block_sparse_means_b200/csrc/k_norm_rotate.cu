// RMS norm of the queries and keys of each head with the rotary position
// embedding in the same pass (sparsepr_norm_rotate in include/sparsepr.h).
//
//   y = x * rsqrt(mean(x^2) + eps) * w,  (a, b) -> (a cos - b sin, a sin + b cos)
//
// A row is held by LPR lanes of a warp, 8 channels (one 16-byte vector of a
// 16-bit type) each: the mean is a butterfly over those lanes, interleaved
// pairs turn inside a lane, and split halves fetch their partner's 8 channels
// from the lane rot / 16 away.  Everything between the load and the one
// rounding at the store is fp32.
//
// Bound by HBM: every row is read and written once.  A thread keeps its token
// through a group of heads, so that the token's angles are read once for the group,
// queries and keys alike, and has NR_HEADS rows in flight.  118,800 tokens x (24 + 24)
// heads, d = 128, inputs changing: 495 to 520 us, 5.7 to 6.0 TB/s, 0.87 to 0.92 of the copy
// bandwidth (487 us on the inputs of the pass before); fp32, 40,000 tokens: 317 us, 6.3 TB/s.
#include <cuda_fp16.h>

#include "spr_internal.cuh"

namespace spr {
namespace {

constexpr int NR_THREADS = 64;  // 118,800 tokens x 24 heads: 32 523 us, 64 487, 128 495, 256 547
constexpr int NR_HEADS = 4;     // heads whose rows a thread has in flight at once (2: 535 us)

struct NrSide {
  const void* x;
  void* y;
  const void* w;
  const int32_t* pos;
  int64_t xs[3], ys[3];
  int H, N;
};
struct NrArgs {
  NrSide side[2];  // 0 queries, 1 keys
  const float *cos, *sin;
  int32_t* status;
  float eps, inv_d;
  int B, d, rot, halves, norm, table_rows, heads_per_group;
  int joint;  // queries and keys have the same tokens and positions: one list of heads
};

// Eight channels as they lie in memory, and as fp32.
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> fetch8(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
// The same for rows that are read once: they leave the L1 to the tables.
template <typename T>
__device__ __forceinline__ Raw<T> stream8(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.v[i].x), "=r"(r.v[i].y), "=r"(r.v[i].z), "=r"(r.v[i].w)
                 : "l"(reinterpret_cast<const uint4*>(p) + i));
  return r;
}
__device__ __forceinline__ void widen(const Raw<bf16>& r, float* f) {
  const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(const Raw<__half>& r, float* f) {
  const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    f[2 * i] = g.x;
    f[2 * i + 1] = g.y;
  }
}
__device__ __forceinline__ void widen(const Raw<float>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(r.v[i].x);
    f[4 * i + 1] = __uint_as_float(r.v[i].y);
    f[4 * i + 2] = __uint_as_float(r.v[i].z);
    f[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* f) {
  widen(fetch8(p), f);
}
__device__ __forceinline__ void store8(bf16* p, const float* f) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                            pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ void store8(__half* p, const float* f) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(float* p, const float* f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Grid: x tiles of tokens, y groups of heads, z batch (and side, where they differ in tokens).
template <typename TI, typename TO, int LPR>
__global__ void __launch_bounds__(NR_THREADS) k_norm_rotate(const __grid_constant__ NrArgs a) {
  after_previous();
  const int b = blockIdx.z % a.B, z = blockIdx.z / a.B;
  const NrSide& s0 = a.side[z];
  const int h0 = blockIdx.y * a.heads_per_group, h1 = h0 + a.heads_per_group;
  const int l = threadIdx.x % LPR, c0 = 8 * l;  // this lane's channels c0 .. c0 + 7
  const int n = blockIdx.x * (NR_THREADS / LPR) + threadIdx.x / LPR;
  if (h0 >= s0.H + (a.joint ? a.side[1].H : 0)) return;
  // lanes without a row or channels stay for the shuffles
  bool live = n < s0.N;
  const bool mine = c0 < a.d;
  // heads hb .. of side s: their rows are on the way while the angles are fetched
  Raw<TI> raw[NR_HEADS];
  auto fetch = [&](const NrSide& s, int hb, int hi) {
    const TI* x = static_cast<const TI*>(s.x) + b * s.xs[0] + (int64_t)n * s.xs[2] + c0;
#pragma unroll
    for (int u = 0; u < NR_HEADS; ++u)
      if (live && mine && hb + u < hi) raw[u] = stream8(x + (hb + u) * s.xs[1]);
  };
  // this group's heads of the queries, then of the keys
  const int lo0 = h0, hi0 = min(h1, s0.H), lo1 = max(h0 - s0.H, 0), hi1 = a.joint ? min(h1 - s0.H, a.side[1].H) : 0;
  const bool has0 = lo0 < hi0;
  fetch(has0 ? s0 : a.side[1], has0 ? lo0 : lo1, has0 ? hi0 : hi1);
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  const int half = a.rot >> 1;
  if (live && a.rot) {
    const int row = s0.pos ? s0.pos[(int64_t)b * s0.N + n] : n;
    if (row < 0 || row >= a.table_rows) {
      if (a.status && l == 0 && h0 == 0 && atomicCAS(a.status, 0, (int)ERR_INDEX) == 0) {
        a.status[1] = b;
        a.status[2] = n;
        a.status[3] = row;
      }
      live = false;
    } else if (c0 < a.rot) {
      if (a.halves) {  // channel c uses pair c mod rot / 2
        const int64_t at = (int64_t)row * half + (c0 < half ? c0 : c0 - half);
        load8(a.cos + at, cs);
        load8(a.sin + at, sn);
      } else {  // channels c0 .. c0 + 7 are pairs c0 / 2 .. c0 / 2 + 3
        const int64_t at = (int64_t)row * half + (c0 >> 1);
        const float4 c = *reinterpret_cast<const float4*>(a.cos + at);
        const float4 d = *reinterpret_cast<const float4*>(a.sin + at);
        cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
        sn[0] = d.x; sn[1] = d.y; sn[2] = d.z; sn[3] = d.w;
      }
    }
  }
  const bool turned = c0 < a.rot, low = c0 < half;
  const int partner = low ? (threadIdx.x & 31) + half / 8 : (threadIdx.x & 31) - half / 8;
  for (int part = has0 ? 0 : 1; part < 2; ++part) {
    const NrSide& s = part ? a.side[1] : s0;
    const int lo = part ? lo1 : lo0, hi = part ? hi1 : hi0;
    if (lo >= hi) break;
    // The weights go into the angles once for all heads: y_c = r (x_c cw_c + x_o sw_c) with
    // o the other channel of the pair, r the row's reciprocal root.
    float w[8], cw[8], sw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if (s.w && mine) load8(static_cast<const TI*>(s.w) + c0, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (a.halves) {
        const float wo = __shfl_sync(0xffffffffu, w[i], partner);
        cw[i] = cs[i] * w[i];
        sw[i] = (low ? -sn[i] : sn[i]) * wo;
      } else {
        cw[i] = cs[i >> 1] * w[i];
        sw[i] = (i & 1 ? sn[i >> 1] : -sn[i >> 1]) * w[i ^ 1];
      }
    }
    TO* y = static_cast<TO*>(s.y) + b * s.ys[0] + (int64_t)n * s.ys[2] + c0;
    for (int hb = lo; hb < hi; hb += NR_HEADS) {
      if (hb > lo || (part && has0)) fetch(s, hb, hi);
#pragma unroll
      for (int u = 0; u < NR_HEADS; ++u) {
        if (hb + u >= hi) break;  // the same for the whole block
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.f;
        if (live && mine) widen(raw[u], f);
        float r = 1.f;
        if (a.norm) {
          float q = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) q = fmaf(f[i], f[i], q);
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
          r = rsqrtf(fmaf(q, a.inv_d, a.eps));
        }
        if (a.halves && a.rot) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float o = __shfl_sync(0xffffffffu, f[i], partner);
            f[i] = turned ? fmaf(o, sw[i], f[i] * cw[i]) * r : f[i] * cw[i] * r;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = f[2 * i], q = f[2 * i + 1];
            f[2 * i] = turned ? fmaf(q, sw[2 * i], p * cw[2 * i]) * r : p * cw[2 * i] * r;
            f[2 * i + 1] = turned ? fmaf(p, sw[2 * i + 1], q * cw[2 * i + 1]) * r : q * cw[2 * i + 1] * r;
          }
        }
        if (live && mine) store8(y + (hb + u) * s.ys[1], f);
      }
    }
  }
}

template <typename TI, typename TO>
cudaError_t launch(NrArgs a, cudaStream_t st) {
  const int lanes = a.d / 8;
  auto go = [&](auto kern, int lpr) {
    const int per = NR_THREADS / lpr;
    const int sides = a.side[1].H && !a.joint ? 2 : 1;
    const int N = sides == 2 ? max(a.side[0].N, a.side[1].N) : a.side[0].N;
    const int H = a.joint ? a.side[0].H + a.side[1].H : max(a.side[0].H, a.side[1].H);
    // A thread takes its token's angles once for a group of heads, NR_HEADS rows
    // at a time; the fewer groups, the fewer times the tables are read.  As many
    // groups as make eight blocks for every SM.
    const int64_t blocks = (int64_t)((N + per - 1) / per) * sides * a.B;
    const int most = (H + NR_HEADS - 1) / NR_HEADS;
    const int64_t need = (8 * num_sms() + blocks - 1) / blocks;
    const int groups = need < most ? (int)need : most;
    a.heads_per_group = ((H + groups - 1) / groups + NR_HEADS - 1) / NR_HEADS * NR_HEADS;
    const dim3 grid((N + per - 1) / per, (H + a.heads_per_group - 1) / a.heads_per_group,
                    sides * a.B);
    spr_launch_early(kern, grid, NR_THREADS, 0, st, a);
    return cudaGetLastError();
  };
  if (lanes > 16) return go(k_norm_rotate<TI, TO, 32>, 32);
  if (lanes > 8) return go(k_norm_rotate<TI, TO, 16>, 16);
  if (lanes > 4) return go(k_norm_rotate<TI, TO, 8>, 8);
  return go(k_norm_rotate<TI, TO, 4>, 4);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Rows on 16 bytes: strides in elements, a multiple of `per` where the dimension has more than one entry.
bool side_strides_ok(const int64_t* s, const int* size, int per, bool out) {
  for (int i = 0; i < 3; ++i) {
    if (s[i] < 0 || (size[i] > 1 && s[i] % per)) return false;
    if (out && size[i] > 1 && s[i] == 0) return false;
  }
  return true;
}

}  // namespace
}  // namespace spr

using namespace spr;

extern "C" spr_status sparsepr_norm_rotate(const spr_norm_rotate_params* p, const void* Q,
                                           const void* K, const void* wq, const void* wk,
                                           const float* cos, const float* sin, int32_t table_rows,
                                           const int32_t* pos_q, const int32_t* pos_k, void* Qo,
                                           void* Ko, int32_t* status, void* stream) {
  if (!p || !Q || !Qo) return SPR_EINVAL;
  const bool keys = p->Hk > 0;
  if (p->B < 1 || p->Hq < 1 || p->Hk < 0 || p->Nq < 1 || (keys && p->Nk < 1)) return SPR_EINVAL;
  if (keys && (!K || !Ko)) return SPR_EINVAL;
  if (p->dtype_in < SPR_BF16 || p->dtype_in > SPR_FP32 || p->dtype_out < SPR_BF16 ||
      p->dtype_out > SPR_FP32)
    return SPR_EINVAL;
  if (p->dtype_out != p->dtype_in && p->dtype_out != SPR_BF16) return SPR_EUNSUPPORTED;
  if (p->d < 1 || p->rot < 0 || p->rot > p->d) return SPR_EINVAL;
  if (p->d % 8 || p->d > 256) return SPR_EUNSUPPORTED;
  if (p->pairing != SPR_PAIR_INTERLEAVED && p->pairing != SPR_PAIR_HALVES) return SPR_EINVAL;
  if (p->rot % (p->pairing == SPR_PAIR_HALVES ? 16 : 8)) return SPR_EUNSUPPORTED;
  if ((p->norm != 0 && p->norm != 1) || !(p->eps >= 0.f) || !isfinite(p->eps)) return SPR_EINVAL;
  if (!p->norm && (wq || (keys && wk))) return SPR_EINVAL;
  if (p->rot) {
    if (!cos || !sin || table_rows < 1) return SPR_EINVAL;
    if ((!pos_q && p->Nq > table_rows) || (keys && !pos_k && p->Nk > table_rows))
      return SPR_EINVAL;
    if (!aligned(cos, 16) || !aligned(sin, 16)) return SPR_EUNSUPPORTED;
  }
  if (p->B > 32767 || p->Hq > 65535 || p->Hk > 65535) return SPR_EUNSUPPORTED;
  // (the last block's threads number tokens past the last)
  if (p->Nq > INT32_MAX - NR_THREADS || (keys && p->Nk > INT32_MAX - NR_THREADS))
    return SPR_EUNSUPPORTED;
  const int nq[3] = {p->B, p->Hq, p->Nq}, nk[3] = {p->B, p->Hk, p->Nk};
  const int pi = p->dtype_in == SPR_FP32 ? 4 : 8, po = p->dtype_out == SPR_FP32 ? 4 : 8;
  if (!side_strides_ok(p->q_strides, nq, pi, false) || !side_strides_ok(p->qo_strides, nq, po, true))
    return SPR_EUNSUPPORTED;
  if (keys && (!side_strides_ok(p->k_strides, nk, pi, false) ||
               !side_strides_ok(p->ko_strides, nk, po, true)))
    return SPR_EUNSUPPORTED;
  if (!aligned(Q, 16) || !aligned(Qo, 16) || !aligned(wq, 16) ||
      (keys && (!aligned(K, 16) || !aligned(Ko, 16) || !aligned(wk, 16))) || !aligned(pos_q, 4) ||
      !aligned(pos_k, 4) || !aligned(status, 4))
    return SPR_EUNSUPPORTED;

  NrArgs a{};
  a.side[0] = {Q, Qo, wq, pos_q, {}, {}, p->Hq, p->Nq};
  if (keys) a.side[1] = {K, Ko, wk, pos_k, {}, {}, p->Hk, p->Nk};
  for (int i = 0; i < 3; ++i) {
    a.side[0].xs[i] = p->q_strides[i];
    a.side[0].ys[i] = p->qo_strides[i];
    a.side[1].xs[i] = p->k_strides[i];
    a.side[1].ys[i] = p->ko_strides[i];
  }
  a.cos = cos;
  a.sin = sin;
  a.status = status;
  a.eps = p->eps;
  a.inv_d = 1.f / (float)p->d;
  a.B = p->B;
  a.d = p->d;
  a.rot = p->rot;
  a.halves = p->pairing == SPR_PAIR_HALVES;
  a.norm = p->norm;
  a.table_rows = table_rows;
  a.joint = keys && p->Nq == p->Nk && pos_q == pos_k;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (status && cudaMemsetAsync(status, 0, 4 * sizeof(int32_t), st) != cudaSuccess)
    return SPR_ECUDA;
  cudaError_t e;
  if (p->dtype_in == SPR_BF16)
    e = launch<bf16, bf16>(a, st);
  else if (p->dtype_in == SPR_FP16)
    e = p->dtype_out == SPR_FP16 ? launch<__half, __half>(a, st) : launch<__half, bf16>(a, st);
  else
    e = p->dtype_out == SPR_FP32 ? launch<float, float>(a, st) : launch<float, bf16>(a, st);
  return e == cudaSuccess ? SPR_OK : SPR_ECUDA;
}
