// Routing of tokens to experts: scores from router logits, the choice of topk experts by
// score + bias within the best groups, and the chosen experts' weights.
#include "common.cuh"
#include "moe.h"

namespace dsv4 {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ double score64(int fn, double l, double mx, double sum) {
  if (fn == DSV4_SCORE_SOFTMAX) return mx == -INFINITY ? 0.0 : exp(l - mx) / sum;
  if (fn == DSV4_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
  return sqrt(log1p(exp(-fabs(l))) + fmax(l, 0.0));
}

__device__ __forceinline__ double warp_sum64(double v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One warp per token; every score in 64 bits.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteArgs a) {
  extern __shared__ double smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
  if (t >= a.T) return;
  double* score = smem + (size_t)warp * 2 * a.E;
  double* choice = score + a.E;  // NaN: not to be chosen any more
  const T* row = static_cast<const T*>(a.logits) + t * a.E;
  double mx = -INFINITY, sum = 0.0;
  if (a.score_fn == DSV4_SCORE_SOFTMAX) {
    for (int e = lane; e < a.E; e += 32) mx = fmax(mx, (double)to_f32<T>(row[e]));
    for (int o = 16; o > 0; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    for (int e = lane; e < a.E; e += 32) sum += exp((double)to_f32<T>(row[e]) - mx);
    sum = warp_sum64(sum);
  }
  for (int e = lane; e < a.E; e += 32) {
    const double s = score64(a.score_fn, (double)to_f32<T>(row[e]), mx, sum);
    const double c = s + (a.bias ? (double)a.bias[e] : 0.0);
    score[e] = s;
    choice[e] = c == c ? c : -INFINITY;
  }
  __syncwarp();
  if (a.n_group > 1) {
    const int per = a.E / a.n_group;
    double best = -INFINITY;
    bool open = lane < a.n_group;
    if (open) {
      double b0 = -INFINITY, b1 = -INFINITY;
      for (int i = 0; i < per; ++i) {
        const double c = choice[lane * per + i];
        if (c > b0) { b1 = b0; b0 = c; } else if (c > b1) { b1 = c; }
      }
      best = per > 1 ? b0 + b1 : b0;
      if (best != best) best = -INFINITY;
    }
    bool kept = false;
    for (int j = 0; j < a.topk_group; ++j) {
      double v = best;
      int at = open && !kept ? lane : 64;
      for (int o = 16; o > 0; o >>= 1) {
        const double v2 = __shfl_xor_sync(0xffffffffu, v, o);
        const int at2 = __shfl_xor_sync(0xffffffffu, at, o);
        if (at2 < 64 && (at == 64 || v2 > v || (v2 == v && at2 < at))) { v = v2; at = at2; }
      }
      if (at == lane) kept = true;
    }
    const unsigned kept_mask = __ballot_sync(0xffffffffu, kept);
    for (int e = lane; e < a.E; e += 32)
      if (!((kept_mask >> (e / per)) & 1u)) choice[e] = nan("");
    __syncwarp();
  }
  double mine = 0.0, total = 0.0;
  int my_id = -1;
  for (int j = 0; j < a.topk; ++j) {
    double v = 0.0;
    int at = 1 << 30;
    for (int e = lane; e < a.E; e += 32) {
      const double c = choice[e];
      if (c == c && (at == 1 << 30 || c > v)) { v = c; at = e; }
    }
    for (int o = 16; o > 0; o >>= 1) {
      const double v2 = __shfl_xor_sync(0xffffffffu, v, o);
      const int at2 = __shfl_xor_sync(0xffffffffu, at, o);
      if (at2 < 1 << 30 && (at == 1 << 30 || v2 > v || (v2 == v && at2 < at))) { v = v2; at = at2; }
    }
    const double s = score[at];
    total += s;
    if (lane == j) { mine = s; my_id = at; }
    __syncwarp();
    if (lane == 0) choice[at] = nan("");
    __syncwarp();
  }
  if (lane < a.topk) {
    a.ids[t * a.topk + lane] = my_id;
    a.weights[t * a.topk + lane] = (float)((a.renorm ? mine / (total + 1e-20) : mine) * (double)a.routed_scale);
  }
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, int dtype, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const int grid = (a.T + kWarps - 1) / kWarps;
  const size_t smem = (size_t)kWarps * 2 * a.E * sizeof(double);
  const void* fn = dtype == DSV4_BF16 ? (const void*)route_kernel<__nv_bfloat16> : (const void*)route_kernel<float>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  if (dtype == DSV4_BF16)
    route_kernel<__nv_bfloat16><<<grid, kWarps * 32, smem, st>>>(a);
  else
    route_kernel<float><<<grid, kWarps * 32, smem, st>>>(a);
  note_launch(1);
  return cudaGetLastError();
}

}  // namespace dsv4
