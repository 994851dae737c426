// Residual addition and root-mean-square norm, with an optional 8-bit form.
//
//   r = x + residual                                    (32 bits)
//   y = r / sqrt(mean(r^2) + eps) * weight
//   s_g = max_{c in group g} |y_c| / 448,  q_c = e4m3(y_c / s_g)     128 channels per group
// r is stored as res_out, y as y, (q, s) as yq / yscale; each is rounded once, from the 32-bit
// value (y is formed from the unrounded r).
#include <cuda_fp8.h>

#include "common.cuh"
#include "moe.h"

namespace dsv4 {
namespace {

__device__ __forceinline__ float group_scale(float amax, int pow2) {
  float s = amax / kE4M3Max;
  if (s == 0.f) return 1.f;  // an all-zero group
  if (pow2 && s < INFINITY) {  // the smallest power of two that is not below it; NaN stays
    int e;
    const float m = frexpf(s, &e);
    s = ldexpf(1.f, m == 0.5f ? e - 1 : e);
  }
  return s;
}

template <typename T>
__global__ void __launch_bounds__(256) norm_kernel(NormArgs a) {
  __shared__ float part[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t base = (int64_t)blockIdx.x * a.hidden;
  const T* x = static_cast<const T*>(a.x) + base;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + base : nullptr;
  const T* w = static_cast<const T*>(a.weight);
  float sq = 0.f;
  for (int c = tid; c < a.hidden; c += 256) {
    const float r = to_f32<T>(x[c]) + (res ? to_f32<T>(res[c]) : 0.f);
    sq += r * r;
  }
  sq = warp_sum(sq);
  if (lane == 0) part[warp] = sq;
  __syncthreads();
  sq = 0.f;
  for (int i = 0; i < 8; ++i) sq += part[i];
  const float inv = rsqrtf(sq / (float)a.hidden + a.eps);
  const int groups = (a.hidden + kScaleGroup - 1) / kScaleGroup;
  for (int g = warp; g < groups; g += 8) {
    float y[4], amax = 0.f;
    bool nan = false;
    for (int i = 0; i < 4; ++i) {
      const int c = g * kScaleGroup + i * 32 + lane;
      y[i] = 0.f;
      if (c >= a.hidden) continue;
      const float r = to_f32<T>(x[c]) + (res ? to_f32<T>(res[c]) : 0.f);
      y[i] = r * inv * to_f32<T>(w[c]);
      if (a.res_out) static_cast<T*>(a.res_out)[base + c] = from_f32<T>(r);
      if (a.y) static_cast<T*>(a.y)[base + c] = from_f32<T>(y[i]);
      amax = fmaxf(amax, fabsf(y[i]));
      nan |= y[i] != y[i];
    }
    if (!a.yq) continue;
    amax = warp_max(amax);
    if (__any_sync(0xffffffffu, nan)) amax = nanf("");
    const float s = group_scale(amax, a.scale_pow2);
    if (lane == 0) a.yscale[(int64_t)blockIdx.x * groups + g] = s;
    for (int i = 0; i < 4; ++i) {
      const int c = g * kScaleGroup + i * 32 + lane;
      if (c < a.hidden) a.yq[base + c] = __nv_cvt_float_to_fp8(y[i] / s, __NV_SATFINITE, __NV_E4M3);
    }
  }
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  if (dtype == DSV4_BF16)
    norm_kernel<__nv_bfloat16><<<a.T, 256, 0, st>>>(a);
  else
    norm_kernel<float><<<a.T, 256, 0, st>>>(a);
  note_launch(1);
  return cudaGetLastError();
}

}  // namespace dsv4
