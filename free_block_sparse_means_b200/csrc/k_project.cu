// Matrix product with its epilogue (sparsepr_project in include/sparsepr.h):
//   Y = R + gate_b * act(X W^T + bias)
// with X, Y and R row-major or head-major.  A 64 x 64 tile of Y per block,
// operands staged in shared memory in fp32, 4 x 4 results per thread.
#include <cuda_fp16.h>

#include "spr_internal.cuh"

namespace spr {
namespace {

struct PjArgs {
  const void *X, *W, *bias, *gate, *R;
  void* Y;
  int64_t xs[3], ys[3], rs[3], ws;
  int B, N, K, M, dx, dy, act;
};

__device__ __forceinline__ float tof(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float tof(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

__device__ __forceinline__ float activate(float x, int act) {
  if (act == SPR_ACT_GELU) return 0.5f * x * (1.f + erff(x * 0.70710678118654752f));
  if (act == SPR_ACT_GELU_TANH)
    return 0.5f * x * (1.f + tanhf(0.79788456080286536f * (x + 0.044715f * x * x * x)));
  if (act == SPR_ACT_SILU) return x / (1.f + expf(-x));
  return x;
}

constexpr int PT = 64, PK = 16;

template <typename T>
__global__ void __launch_bounds__(256) k_project_simple(const __grid_constant__ PjArgs a) {
  __shared__ float sx[PK][PT + 1], sw[PK][PT + 1];
  const int b = blockIdx.z, n0 = blockIdx.y * PT, m0 = blockIdx.x * PT;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const T* X = static_cast<const T*>(a.X) + b * a.xs[0];
  const T* W = static_cast<const T*>(a.W);
  float acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += PK) {
    for (int i = threadIdx.x; i < PT * PK; i += 256) {
      const int r = i / PK, k = i % PK, kk = k0 + k;
      float x = 0.f, w = 0.f;
      if (kk < a.K && n0 + r < a.N)
        x = tof(X[(int64_t)(n0 + r) * a.xs[2] + (kk / a.dx) * a.xs[1] + kk % a.dx]);
      if (kk < a.K && m0 + r < a.M) w = tof(W[(int64_t)(m0 + r) * a.ws + kk]);
      sx[k][r] = x;
      sw[k][r] = w;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sx[k][ty + 16 * i], sw[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + ty + 16 * i, m = m0 + tx + 16 * j;
      if (n >= a.N || m >= a.M) continue;
      float v = acc[i][j];
      if (a.bias) v += tof(static_cast<const T*>(a.bias)[m]);
      v = activate(v, a.act);
      if (a.gate) v *= tof(static_cast<const T*>(a.gate)[(int64_t)b * a.M + m]);
      if (a.R)
        v += tof(static_cast<const T*>(
            a.R)[b * a.rs[0] + (m / a.dy) * a.rs[1] + (int64_t)n * a.rs[2] + m % a.dy]);
      put(static_cast<T*>(a.Y) + b * a.ys[0] + (m / a.dy) * a.ys[1] + (int64_t)n * a.ys[2] + m % a.dy,
          v);
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool strides_fit(const int64_t* s, int B, int H, int N, bool out) {
  const int size[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    if (s[i] < 0 || (size[i] > 1 && s[i] % 8)) return false;
    if (out && size[i] > 1 && s[i] == 0) return false;
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

}  // namespace
}  // namespace spr

using namespace spr;

extern "C" size_t sparsepr_project_workspace(const spr_project_params* p) {
  return check(p) == SPR_OK ? 256 : 0;
}

extern "C" spr_status sparsepr_project(const spr_project_params* p, const void* X, const void* W,
                                       const void* bias, const void* gate, const void* R, void* Y,
                                       void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  const spr_status s = check(p);
  if (s != SPR_OK) return s;
  if (!X || !W || !Y) return SPR_EINVAL;
  if (!ws || !aligned(ws, 256) || ws_bytes < sparsepr_project_workspace(p)) return SPR_EWORKSPACE;
  if (!aligned(X, 16) || !aligned(W, 16) || !aligned(Y, 16) || !aligned(R, 16) ||
      !aligned(bias, 16) || !aligned(gate, 16) || !aligned(status, 4))
    return SPR_EUNSUPPORTED;
  if (R && !strides_fit(p->r_strides, p->B, p->Hy, p->N, false)) return SPR_EUNSUPPORTED;
  PjArgs a{X, W, bias, gate, R, Y, {}, {}, {}, p->w_stride, p->B, p->N, p->Hx * p->dx,
           p->Hy * p->dy, p->dx, p->dy, p->act};
  for (int i = 0; i < 3; ++i) {
    a.xs[i] = p->x_strides[i];
    a.ys[i] = p->y_strides[i];
    a.rs[i] = p->r_strides[i];
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (status && cudaMemsetAsync(status, 0, 4 * sizeof(int32_t), st) != cudaSuccess)
    return SPR_ECUDA;
  const dim3 grid((a.M + PT - 1) / PT, (a.N + PT - 1) / PT, a.B);
  if (p->dtype == SPR_BF16)
    spr_launch(k_project_simple<bf16>, grid, 256, 0, st, a);
  else
    spr_launch(k_project_simple<__half>, grid, 256, 0, st, a);
  return cudaGetLastError() == cudaSuccess ? SPR_OK : SPR_ECUDA;
}
