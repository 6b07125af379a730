// Exact attention under a mask (sparsepr_attend_masked in include/sparsepr.h).
// One block per (batch, head, 32 queries): keys pass through shared memory 32
// at a time, each warp keeps 4 query rows with their running maximum, sum and
// output, each lane one key's score and d / 32 output channels.
#include <cuda_fp16.h>

#include "spr_internal.cuh"

namespace spr {
namespace {

struct AmArgs {
  const void *Q, *K, *V;
  void* O;
  float* lse;
  const int32_t *k_len, *doc_q, *doc_k, *prefix;
  const float* slopes;
  int64_t qs[3], ks[3], vs[3], os[3];
  int B, Hq, Hk, Nq, Nk, causal, q_start;
  float scale, softcap;
};

__device__ __forceinline__ float tof(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float tof(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

template <typename T, int D>
__global__ void __launch_bounds__(256) k_attend_simple(const __grid_constant__ AmArgs a) {
  __shared__ float sk[32][D + 1];
  __shared__ T sv[32][D];
  __shared__ float sq[32][D];
  const int b = blockIdx.z, h = blockIdx.y, i0 = blockIdx.x * 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = h / (a.Hq / a.Hk);
  const T* Q = static_cast<const T*>(a.Q) + b * a.qs[0] + h * a.qs[1];
  const T* K = static_cast<const T*>(a.K) + b * a.ks[0] + hk * a.ks[1];
  const T* V = static_cast<const T*>(a.V) + b * a.vs[0] + hk * a.vs[1];
  const int len = a.k_len ? min(max(a.k_len[b], 0), a.Nk) : a.Nk;
  const int pos0 = a.q_start == SPR_ALIGN_END ? len - a.Nq : a.q_start;
  const int pre = a.prefix ? a.prefix[b] : 0;
  for (int i = threadIdx.x; i < 32 * D; i += 256)
    sq[i / D][i % D] = i0 + i / D < a.Nq ? tof(Q[(int64_t)(i0 + i / D) * a.qs[2] + i % D]) : 0.f;
  float m[4], l[4], o[4][D / 32];
  for (int r = 0; r < 4; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
    for (int c = 0; c < D / 32; ++c) o[r][c] = 0.f;
  }
  for (int j0 = 0; j0 < len; j0 += 32) {
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * D; i += 256) {
      const int j = j0 + i / D;
      const bool dead = j >= len || (a.doc_k && a.doc_k[(int64_t)b * a.Nk + j] < 0);
      sk[i / D][i % D] = dead ? 0.f : tof(K[(int64_t)j * a.ks[2] + i % D]);
      sv[i / D][i % D] = dead ? T(0.f) : V[(int64_t)j * a.vs[2] + i % D];
    }
    __syncthreads();
    const int j = j0 + lane;
    const int dk = a.doc_k && j < len ? a.doc_k[(int64_t)b * a.Nk + j] : 0;
    for (int r = 0; r < 4; ++r) {
      const int i = i0 + 4 * warp + r;
      float x = 0.f;
      for (int c = 0; c < D; ++c) x = fmaf(sq[4 * warp + r][c], sk[lane][c], x);
      x *= a.scale;
      if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
      const int p = pos0 + i;
      if (a.slopes) x -= a.slopes[h] * fabsf((float)(p - j));
      bool see = i < a.Nq && j < len;
      if (a.doc_k) see = see && dk >= 0 && a.doc_q[(int64_t)b * a.Nq + min(i, a.Nq - 1)] == dk;
      if (a.causal) see = see && (j <= p || j < pre);
      if (!see) x = -INFINITY;
      const float mn = fmaxf(m[r], warp_max(x));
      const float ms = mn == -INFINITY ? 0.f : mn;
      const float e = expf(x - ms), corr = expf(m[r] - ms);
      l[r] = l[r] * corr + warp_sum(e);
      m[r] = mn;
      for (int c = 0; c < D / 32; ++c) o[r][c] *= corr;
      for (int k = 0; k < 32; ++k) {
        const float w = __shfl_sync(0xffffffffu, e, k);
        for (int c = 0; c < D / 32; ++c) o[r][c] = fmaf(w, tof(sv[k][lane + 32 * c]), o[r][c]);
      }
    }
  }
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + 4 * warp + r;
    if (i >= a.Nq) break;
    T* O = static_cast<T*>(a.O) + b * a.os[0] + h * a.os[1] + (int64_t)i * a.os[2];
    const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
    for (int c = 0; c < D / 32; ++c) put(O + lane + 32 * c, o[r][c] * inv);
    if (a.lse && lane == 0)
      a.lse[((int64_t)b * a.Hq + h) * a.Nq + i] = l[r] > 0.f ? m[r] + logf(l[r]) : -INFINITY;
  }
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
  if (p->Nq > (1 << 30) || p->Nk > (1 << 30) || p->B > 65535 || p->Hq > 65535)
    return SPR_EUNSUPPORTED;
  if (!strides_fit(p->q_strides, p->B, p->Hq, p->Nq, false) ||
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
  return check(p) == SPR_OK ? 256 : 0;
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
  AmArgs a{Q, K, V, O, lse, k_len, doc_q, doc_k, prefix, slopes, {}, {}, {}, {}, p->B, p->Hq, p->Hk,
           p->Nq, p->Nk, p->causal, p->q_start, 0.f, p->softcap};
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = p->q_strides[i];
    a.ks[i] = p->k_strides[i];
    a.vs[i] = p->v_strides[i];
    a.os[i] = p->o_strides[i];
  }
  a.scale = p->scale > 0.f ? p->scale : 1.f / sqrtf((float)p->d);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (status && cudaMemsetAsync(status, 0, 4 * sizeof(int32_t), st) != cudaSuccess)
    return SPR_ECUDA;
  const dim3 grid((a.Nq + 31) / 32, a.Hq, a.B);
  auto go = [&](auto kern) { spr_launch(kern, grid, 256, 0, st, a); };
  if (p->dtype == SPR_BF16)
    p->d == 64 ? go(k_attend_simple<bf16, 64>) : go(k_attend_simple<bf16, 128>);
  else
    p->d == 64 ? go(k_attend_simple<__half, 64>) : go(k_attend_simple<__half, 128>);
  return cudaGetLastError() == cudaSuccess ? SPR_OK : SPR_ECUDA;
}
