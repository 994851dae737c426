// Launchers of the operators that follow the attention in a decoder layer (norm.cu, route.cu,
// experts.cu).  Arguments arrive validated, T > 0; each launcher returns the cudaGetLastError() of its
// launches.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dsv4.h"

namespace dsv4 {

void note_launch(int n);

constexpr int kScaleGroup = 128;       // channels that share a scale of the 8-bit form
constexpr float kE4M3Max = 448.f;      // largest finite e4m3 value
constexpr int kMaxWidth = 1 << 20;      // channels of a row
constexpr int kMaxExperts = 1024;
constexpr int kMaxRouteTopk = 32;
constexpr int kMaxRouteGroups = 32;
constexpr int kMaxExpertTopk = 64;

struct NormArgs {
  int T, hidden, scale_pow2;
  float eps;
  const void* x;
  const void* residual;  // may be NULL
  const void* weight;
  void* res_out;         // may be NULL; may be x or residual
  void* y;               // may be NULL; may be x or residual
  uint8_t* yq;           // may be NULL
  float* yscale;
};
cudaError_t launch_norm(const NormArgs& a, int dtype, cudaStream_t st);

struct RouteArgs {
  int T, E, topk, n_group, topk_group, score_fn, renorm;
  float routed_scale;
  const void* logits;
  const float* bias;  // may be NULL
  int32_t* ids;
  float* weights;
};
cudaError_t launch_route(const RouteArgs& a, int dtype, cudaStream_t st);

struct ExpertArgs {
  int T, hidden, inter, E, topk;
  float limit;           // 0: no clamp
  const void* x;         // [T, hidden] bf16, or e4m3 with x_scale
  const float* x_scale;  // [T, ceil(hidden/128)] or NULL
  const int32_t* ids;
  const float* weights;
  const void* w13;
  const void* w2;
  void* out;
  void* ws;
};
size_t expert_workspace_bytes(int64_t T, int hidden, int inter, int E, int topk);
cudaError_t launch_experts(const ExpertArgs& a, cudaStream_t st);
cudaError_t take_experts_error(int* code);

}  // namespace dsv4
