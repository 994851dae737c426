// The experts' products of a routed layer:
//   out[t] = sum_j weights[t,j] * W2_e h,  h = silu(g) * u,  g = W1_e x_t,  u = W3_e x_t,  e = ids[t,j]
// with g <- min(g, limit) and u <- clamp(u, -limit, limit) when a limit is given.
// The (token, choice) pairs are put in order of their expert; h is rounded to bf16 (the type of
// the second product's operands), the products of a pair are kept in 32 bits until the sum over j.
#include <cuda_fp8.h>

#include "common.cuh"
#include "moe.h"

namespace dsv4 {
namespace {

constexpr int kTile = 64, kStep = 16;

struct Layout {
  size_t offs, row_slot, slot_row, h, yp, total;
};
Layout layout(int64_t T, int hidden, int inter, int E, int topk) {
  const int64_t n = T * topk;
  Layout l{};
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  l.offs = 0;
  l.row_slot = up((size_t)(E + 1) * 4);
  l.slot_row = l.row_slot + up((size_t)n * 4);
  l.h = l.slot_row + up((size_t)n * 4);
  l.yp = l.h + up((size_t)n * inter * 2);
  l.total = l.yp + up((size_t)n * hidden * 4);
  return l;
}

// One CTA: rows of the pairs in order of their expert.
__global__ void __launch_bounds__(1024) order_kernel(const int32_t* ids, int64_t n, int E, int32_t* offs,
                                                     int32_t* row_slot, int32_t* slot_row) {
  __shared__ int32_t count[kMaxExperts], at[kMaxExperts];
  for (int e = threadIdx.x; e < E; e += blockDim.x) count[e] = 0;
  __syncthreads();
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
    const int e = ids[i];
    if (e >= 0 && e < E) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int s = 0;
    for (int e = 0; e < E; ++e) {
      offs[e] = at[e] = s;
      s += count[e];
    }
    offs[E] = s;
  }
  __syncthreads();
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
    const int e = ids[i];
    int r = -1;
    if (e >= 0 && e < E) {
      r = atomicAdd(&at[e], 1);
      row_slot[r] = (int32_t)i;
    }
    slot_row[i] = r;
  }
}

// 64 rows x 64 columns of one expert's product, blockIdx.z the expert.
template <int kPass>
__global__ void __launch_bounds__(256) product_kernel(ExpertArgs a, const int32_t* offs, const int32_t* row_slot,
                                                      __nv_bfloat16* h, float* yp) {
  __shared__ float sa[kStep][kTile], sb[kStep][kTile], sc[kStep][kTile];
  const int e = blockIdx.z, r0 = offs[e], n = offs[e + 1] - r0;
  const int c0 = blockIdx.x * kTile, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int K = kPass == 0 ? a.hidden : a.inter, N = kPass == 0 ? a.inter : a.hidden;
  const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(kPass == 0 ? a.w13 : a.w2) +
                           (int64_t)e * N * K * (kPass == 0 ? 2 : 1);
  for (int m0 = blockIdx.y * kTile; m0 < n; m0 += gridDim.y * kTile) {
    float acc[4][4] = {}, acc2[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += kStep) {
      for (int i = tid; i < kTile * kStep; i += 256) {
        const int kk = i % kStep, m = i / kStep, k = k0 + kk;
        float v = 0.f;
        if (m0 + m < n && k < K) {
          const int64_t row = r0 + m0 + m;
          if (kPass == 0) {
            const int64_t t = row_slot[row] / a.topk;
            if (a.x_scale) {
              const __nv_fp8_e4m3 q = static_cast<const __nv_fp8_e4m3*>(a.x)[t * K + k];
              v = (float)q * a.x_scale[t * ((K + kScaleGroup - 1) / kScaleGroup) + k / kScaleGroup];
            } else {
              v = __bfloat162float(static_cast<const __nv_bfloat16*>(a.x)[t * K + k]);
            }
          } else {
            v = __bfloat162float(h[row * K + k]);
          }
        }
        sa[kk][m] = v;
        const bool in = c0 + m < N && k < K;
        sb[kk][m] = in ? __bfloat162float(w[(int64_t)(c0 + m) * K + k]) : 0.f;
        if (kPass == 0) sc[kk][m] = in ? __bfloat162float(w[(int64_t)(N + c0 + m) * K + k]) : 0.f;
      }
      __syncthreads();
      for (int kk = 0; kk < kStep; ++kk)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) {
            acc[i][j] += sa[kk][ty * 4 + i] * sb[kk][tx + 16 * j];
            if (kPass == 0) acc2[i][j] += sa[kk][ty * 4 + i] * sc[kk][tx + 16 * j];
          }
      __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int m = m0 + ty * 4 + i, c = c0 + tx + 16 * j;
        if (m >= n || c >= N) continue;
        const int64_t row = r0 + m;
        if (kPass == 0) {
          float g = acc[i][j], u = acc2[i][j];
          if (a.limit > 0.f) {
            g = g > a.limit ? a.limit : g;  // a NaN stays one
            u = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
          }
          h[row * N + c] = __float2bfloat16_rn(g / (1.f + __expf(-g)) * u);
        } else {
          yp[row * N + c] = acc[i][j] * a.weights[row_slot[row]];
        }
      }
  }
}

__global__ void __launch_bounds__(256) combine_kernel(ExpertArgs a, const int32_t* slot_row, const float* yp) {
  const int64_t t = blockIdx.x;
  for (int c = threadIdx.x; c < a.hidden; c += 256) {
    float s = 0.f;
    for (int j = 0; j < a.topk; ++j) {
      const int r = slot_row[t * a.topk + j];
      if (r >= 0) s += yp[(int64_t)r * a.hidden + c];
    }
    static_cast<__nv_bfloat16*>(a.out)[t * a.hidden + c] = __float2bfloat16_rn(s);
  }
}

}  // namespace

size_t expert_workspace_bytes(int64_t T, int hidden, int inter, int E, int topk) {
  return layout(T, hidden, inter, E, topk).total;
}

cudaError_t launch_experts(const ExpertArgs& a, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const Layout l = layout(a.T, a.hidden, a.inter, a.E, a.topk);
  char* ws = static_cast<char*>(a.ws);
  int32_t* offs = reinterpret_cast<int32_t*>(ws + l.offs);
  int32_t* row_slot = reinterpret_cast<int32_t*>(ws + l.row_slot);
  int32_t* slot_row = reinterpret_cast<int32_t*>(ws + l.slot_row);
  __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(ws + l.h);
  float* yp = reinterpret_cast<float*>(ws + l.yp);
  const int64_t n = (int64_t)a.T * a.topk;
  order_kernel<<<1, 1024, 0, st>>>(a.ids, n, a.E, offs, row_slot, slot_row);
  const int64_t want = (n + kTile - 1) / kTile;
  const unsigned my = (unsigned)(want < 64 ? want : 64);
  product_kernel<0><<<dim3((a.inter + kTile - 1) / kTile, my, a.E), 256, 0, st>>>(a, offs, row_slot, h, yp);
  product_kernel<1><<<dim3((a.hidden + kTile - 1) / kTile, my, a.E), 256, 0, st>>>(a, offs, row_slot, h, yp);
  combine_kernel<<<a.T, 256, 0, st>>>(a, slot_row, yp);
  note_launch(4);
  return cudaGetLastError();
}

}  // namespace dsv4
