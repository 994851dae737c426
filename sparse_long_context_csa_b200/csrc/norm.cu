// Residual addition and root-mean-square norm, with an optional 8-bit form.
//
//   r = x + residual                                    (32 bits)
//   y = r / sqrt(mean(r^2) + eps) * weight
//   s_g = max_{c in group g} |y_c| / 448,  q_c = e4m3(y_c / s_g)     128 channels per group
// r is stored as res_out, y as y, (q, s) as yq / yscale; each is rounded once, from the 32-bit
// value (y is formed from the unrounded r).
//
// Bound by memory: every row is read once, kept in registers in 32 bits over the one reduction,
// and written once.  A lane's pieces are 16 bytes (8 bf16 or 4 fp32 channels), so that the 128
// channels of a scale lie in 16 or 32 neighbouring lanes.
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.cuh"
#include "moe.h"

namespace dsv4 {
namespace {

__device__ __forceinline__ float group_scale(float amax, int pow2) {
  float s = amax / kE4M3Max;
  if (s == 0.f) return 1.f;        // an all-zero group
  if (pow2 && s < INFINITY) {      // the smallest power of two that is not below it; NaN stays
    int e;
    const float m = frexpf(s, &e);
    s = ldexpf(1.f, m == 0.5f ? e - 1 : e);
  }
  return s;
}

// v / s.  A power of two within fp32's normal range has an exact reciprocal; of another scale the product
// with its rounded reciprocal is brought to the quotient by its remainder (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990); the sign is that of the product,
// for a zero's.  8191 x 4096 bf16: 49.0 us, by `/` 51.5, by the rounded reciprocal alone 48.3, which put two of
// eight million values a step beside e4m3(v / s).
template <int kN>
__device__ __forceinline__ void divide(float (&v)[kN], float s, int pow2) {
  if (s >= 0x1p-100f && s < INFINITY) {
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const float q = v[j] * inv;
      v[j] = pow2 ? q : copysignf(fmaf(fmaf(-q, s, v[j]), inv, q), q);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] /= s;
  }
}

template <typename T>
struct Piece;  // 16 bytes of a row
template <>
struct Piece<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint4 v;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return v;
  }
};

// `per` threads (a multiple of 32) have a row, kV pieces each; rows of one warp share a CTA, wider
// ones have it to themselves.
template <typename T, int kV>
__global__ void __launch_bounds__(1024) norm_rows_kernel(NormArgs a, int per) {
  constexpr int kN = Piece<T>::kN;
  __shared__ float part[32];
  const int lane = threadIdx.x & 31, i0 = per == 32 ? lane : threadIdx.x;
  const int64_t row = per == 32 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  const int n = a.hidden / kN;
  const uint4* w = static_cast<const uint4*>(a.weight);
  wait_for_previous();
  if (row >= a.T) return;
  const uint4* x = static_cast<const uint4*>(a.x) + row * n;
  const uint4* res = a.residual ? static_cast<const uint4*>(a.residual) + row * n : nullptr;
  uint4 vx[kV], vr[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int i = i0 + v * per;
    vx[v] = vr[v] = make_uint4(0, 0, 0, 0);
    if (i < n) {
      vx[v] = x[i];
      if (res) vr[v] = res[i];
    }
  }
  float r[kV][kN];
  float sq = 0.f;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    float f[kN];
    Piece<T>::unpack(vx[v], r[v]);
    Piece<T>::unpack(vr[v], f);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      r[v][j] += f[j];
      sq = fmaf(r[v][j], r[v][j], sq);
    }
  }
  if (a.res_out) {
    uint4* out = static_cast<uint4*>(a.res_out) + row * n;
#pragma unroll
    for (int v = 0; v < kV; ++v)
      if (i0 + v * per < n) out[i0 + v * per] = Piece<T>::pack(r[v]);
  }
  sq = warp_sum(sq);
  if (per > 32) {
    if (lane == 0) part[threadIdx.x >> 5] = sq;
    __syncthreads();
    sq = warp_sum(lane < (per >> 5) ? part[lane] : 0.f);
  }
  const float inv_rms = rsqrtf(sq / (float)a.hidden + a.eps);
  const int groups = (a.hidden + kScaleGroup - 1) / kScaleGroup;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int i = i0 + v * per;
    float f[kN];
    Piece<T>::unpack(i < n ? w[i] : make_uint4(0, 0, 0, 0), f);
#pragma unroll
    for (int j = 0; j < kN; ++j) r[v][j] = r[v][j] * inv_rms * f[j];
    if (a.y && i < n) static_cast<uint4*>(a.y)[row * n + i] = Piece<T>::pack(r[v]);
    if (!a.yq) continue;
    uint32_t most = 0;  // of the magnitudes' bits: a NaN is above infinity
#pragma unroll
    for (int j = 0; j < kN; ++j) most = max(most, __float_as_uint(r[v][j]) & 0x7fffffffu);
#pragma unroll
    for (int o = kScaleGroup / kN / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    const float s = group_scale(__uint_as_float(i < n ? most : 0u), a.scale_pow2);
    if (i >= n) continue;
    divide(r[v], s, a.scale_pow2);
    if (i % (kScaleGroup / kN) == 0) a.yscale[row * groups + i / (kScaleGroup / kN)] = s;
    uint32_t q[kN / 4];
#pragma unroll
    for (int j = 0; j < kN; j += 4) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(r[v][j], r[v][j + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(r[v][j + 2], r[v][j + 3]), __NV_SATFINITE, __NV_E4M3);
      q[j / 4] = lo | (hi << 16);
    }
    uint8_t* out = a.yq + (row * n + i) * kN;
    if (kN == 8)
      *reinterpret_cast<uint2*>(out) = make_uint2(q[0], q[kN / 4 - 1]);
    else
      *reinterpret_cast<uint32_t*>(out) = q[0];
  }
}

// Rows that are not whole 16-byte pieces, without the 8-bit form.  Behind its first `head` channels a
// row is on a 16-byte boundary: n pieces are read and written whole, the channels before and
// behind them by a thread each.  A CTA (or, with `per` = 32, a warp) takes every stride-th row, a
// multiple of kN, so that its rows have one head and its weights stay in registers; the next row
// is on its way while one is finished.
constexpr int kShiftThreads = 512;
// Threads that an SM is given: half of what it holds, so that a CTA takes several rows (16384 x 1111 bf16 27.7 us,
// 3001 x 1111 fp32 7.9 us with residuals; with 1536 threads 33.6 and 8.9, with 2048 29.2 and 8.7).
constexpr int kShiftHeld = 1024;
template <typename T, int kV>
__global__ void __launch_bounds__(kShiftThreads) norm_shift_kernel(NormArgs a, int per) {
  constexpr int kN = Piece<T>::kN;
  __shared__ float part[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i0 = per == 32 ? lane : threadIdx.x;
  const int rows = per == 32 ? blockDim.x >> 5 : 1;
  const int64_t stride = (int64_t)gridDim.x * rows;
  int64_t row = (int64_t)blockIdx.x * rows + (per == 32 ? warp : 0);
  const int b = (int)(row * a.hidden % kN), head = min((kN - b) % kN, a.hidden);
  const int n = (a.hidden - head) / kN, behind = head + n * kN;
  // this thread's channel outside the pieces: threads 0 .. kN - 1 before them, the next kN behind
  int alone = i0 < kN ? i0 : behind + i0 - kN;
  if (i0 < kN ? i0 >= head : i0 >= 2 * kN || alone >= a.hidden) alone = -1;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  wait_for_previous();
  float w[kV][kN], w_alone = alone >= 0 ? to_f32<T>(static_cast<const T*>(a.weight)[alone]) : 0.f;
#pragma unroll
  for (int v = 0; v < kV; ++v)
#pragma unroll
    for (int j = 0; j < kN; ++j)
      w[v][j] = i0 + v * per < n ? to_f32<T>(static_cast<const T*>(a.weight)[head + (i0 + v * per) * kN + j]) : 0.f;
  uint4 vx[kV], vr[kV];
  T ax = from_f32<T>(0.f), ar = ax;
  auto load = [&](int64_t at) {
    const int64_t base = at * a.hidden;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      vx[v] = vr[v] = make_uint4(0, 0, 0, 0);
      if (i0 + v * per >= n) continue;
      vx[v] = reinterpret_cast<const uint4*>(x + base + head)[i0 + v * per];
      if (res) vr[v] = reinterpret_cast<const uint4*>(res + base + head)[i0 + v * per];
    }
    if (alone >= 0) {
      ax = x[base + alone];
      if (res) ar = res[base + alone];
    }
  };
  auto store = [&](void* out, int64_t base, const float (*f)[kN], float f_alone) {
    T* p = static_cast<T*>(out) + base;
#pragma unroll
    for (int v = 0; v < kV; ++v)
      if (i0 + v * per < n) reinterpret_cast<uint4*>(p + head)[i0 + v * per] = Piece<T>::pack(f[v]);
    if (alone >= 0) p[alone] = from_f32<T>(f_alone);
  };
  if (row < a.T) load(row);
  for (int turn = 0; row < a.T; row += stride, turn ^= 1) {
    const int64_t base = row * a.hidden;
    float r[kV][kN], r_alone = to_f32<T>(ax) + to_f32<T>(ar), sq = r_alone * r_alone;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      float f[kN];
      Piece<T>::unpack(vx[v], r[v]);
      Piece<T>::unpack(vr[v], f);
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        r[v][j] += f[j];
        sq = fmaf(r[v][j], r[v][j], sq);
      }
    }
    if (row + stride < a.T) load(row + stride);
    if (a.res_out) store(a.res_out, base, r, r_alone);
    sq = warp_sum(sq);
    if (per > 32) {  // the other half of `part` is read by whoever is still at the row before
      if (lane == 0) part[turn][warp] = sq;
      __syncthreads();
      sq = warp_sum(lane < (per >> 5) ? part[turn][lane] : 0.f);
    }
    const float inv_rms = rsqrtf(sq / (float)a.hidden + a.eps);
#pragma unroll
    for (int v = 0; v < kV; ++v)
#pragma unroll
      for (int j = 0; j < kN; ++j) r[v][j] = r[v][j] * inv_rms * w[v][j];
    store(a.y, base, r, r_alone * inv_rms * w_alone);
  }
}

// Any width, element by element (with the 8-bit form, and rows too wide for the kernel above): a
// warp has whole groups of 128 channels, four per lane.  kG > 0: at most kG groups per warp, kept in
// registers over the reduction; 0: the row is read a second time.  kW of a CTA's eight warps have a
// row.
template <typename T, int kG, int kW>
__global__ void __launch_bounds__(256) norm_any_kernel(NormArgs a) {
  __shared__ float part[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w0 = warp % kW;
  const int64_t asked = (int64_t)blockIdx.x * (8 / kW) + warp / kW;
  const bool live = asked < a.T;  // a warp without a row goes along with the last one's, for the barrier
  const int64_t row = live ? asked : a.T - 1, base = row * a.hidden;
  const T* x = static_cast<const T*>(a.x) + base;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + base : nullptr;
  const T* w = static_cast<const T*>(a.weight);
  wait_for_previous();
  const int groups = (a.hidden + kScaleGroup - 1) / kScaleGroup;
  auto load = [&](int g, float* r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = g * kScaleGroup + i * 32 + lane;
      r[i] = 0.f;
      if (c < a.hidden) r[i] = to_f32<T>(x[c]) + (res ? to_f32<T>(res[c]) : 0.f);
    }
  };
  constexpr int kHeld = kG > 0 ? kG : 1;
  float r[kHeld][4], sq = 0.f;
  if (kG > 0) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k) load(w0 + k * kW, r[k]);  // zero past the row
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) sq = fmaf(r[k][i], r[k][i], sq);
  } else {
#pragma unroll 2
    for (int g = w0; g < groups; g += kW) {
      load(g, r[0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) sq = fmaf(r[0][i], r[0][i], sq);
    }
  }
  sq = warp_sum(sq);
  if (kW > 1) {
    if (lane == 0) part[warp] = sq;
    __syncthreads();
    sq = 0.f;
#pragma unroll
    for (int i = 0; i < kW; ++i) sq += part[warp - w0 + i];
  }
  if (!live) return;
  const float inv_rms = rsqrtf(sq / (float)a.hidden + a.eps);
  auto finish = [&](int g, float (&v)[4]) {
    uint32_t most = 0;  // of the magnitudes' bits: a NaN is above infinity
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = g * kScaleGroup + i * 32 + lane;
      if (c >= a.hidden) continue;
      if (a.res_out) static_cast<T*>(a.res_out)[base + c] = from_f32<T>(v[i]);
      v[i] = v[i] * inv_rms * to_f32<T>(w[c]);
      if (a.y) static_cast<T*>(a.y)[base + c] = from_f32<T>(v[i]);
      most = max(most, __float_as_uint(v[i]) & 0x7fffffffu);
    }
    if (!a.yq) return;
    const float s = group_scale(__uint_as_float(__reduce_max_sync(0xffffffffu, most)), a.scale_pow2);
    if (lane == 0) a.yscale[row * groups + g] = s;
    divide(v, s, a.scale_pow2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = g * kScaleGroup + i * 32 + lane;
      if (c < a.hidden) a.yq[base + c] = __nv_cvt_float_to_fp8(v[i], __NV_SATFINITE, __NV_E4M3);
    }
  };
  if (kG > 0) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (w0 + k * kW < groups) finish(w0 + k * kW, r[k]);
  } else {
    for (int g = w0; g < groups; g += kW) {
      load(g, r[0]);
      finish(g, r[0]);
    }
  }
}

template <typename T, int kV>
cudaError_t launch_shift(const NormArgs& a, cudaStream_t st) {
  const int n = a.hidden / Piece<T>::kN, per = n <= 32 * kV ? 32 : ((n + kV - 1) / kV + 31) / 32 * 32, rows = per == 32 ? 8 : 1;
  const int64_t blocks = ((int64_t)a.T + rows - 1) / rows, held = (int64_t)sm_count() * (kShiftHeld / (per * rows)) / 8 * 8;
  return launch(norm_shift_kernel<T, kV>, blocks < held ? blocks : held, per * rows, 0, st, a, per);
}

template <typename T>
cudaError_t launch_any(const NormArgs& a, cudaStream_t st) {
  // Without the 8-bit form: as few pieces a thread as there are threads for, up to 16 channels
  // (16384 x 1111 bf16 with a residual: 28.0 us with one, 31.8 with two; element by element 45.8;
  // 4000 x 12001, of 32 channels a thread: 156 us, element by element 136).
  const int n = a.hidden / Piece<T>::kN;
  if (!a.yq && n <= kShiftThreads) return launch_shift<T, 1>(a, st);
  if (!a.yq && n <= 2 * kShiftThreads) return launch_shift<T, 2>(a, st);
  if (!a.yq && n <= 4 * kShiftThreads && sizeof(T) == 4) return launch_shift<T, 4>(a, st);
  // With it, up to 2048 channels the row stays in registers (16384 x 333 bf16: 19.2 us, 36.2 in two
  // passes of a CTA per row; 16384 x 1111: 58.1 and 70.1 us).
  if (a.hidden <= 4 * kScaleGroup) return launch(norm_any_kernel<T, 4, 1>, ((int64_t)a.T + 7) / 8, 256, 0, st, a);
  if (a.hidden <= 8 * kScaleGroup) return launch(norm_any_kernel<T, 4, 2>, ((int64_t)a.T + 3) / 4, 256, 0, st, a);
  if (a.hidden <= 16 * kScaleGroup) return launch(norm_any_kernel<T, 2, 8>, a.T, 256, 0, st, a);
  return launch(norm_any_kernel<T, 0, 8>, a.T, 256, 0, st, a);
}

template <typename T, int kV>
cudaError_t launch_rows(const NormArgs& a, cudaStream_t st) {
  const int n = a.hidden / Piece<T>::kN, per = ((n + kV - 1) / kV + 31) / 32 * 32;
  const int rows = per == 32 ? 8 : 1;  // rows of a CTA
  return launch(norm_rows_kernel<T, kV>, ((int64_t)a.T + rows - 1) / rows, per * rows, 0, st, a, per);
}

template <typename T>
cudaError_t launch_type(const NormArgs& a, cudaStream_t st) {
  const int n = a.hidden / Piece<T>::kN;
  if (a.hidden % Piece<T>::kN != 0 || n > 4096) return launch_any<T>(a, st);
  // Many rows: four pieces a thread, which keeps 128 bytes (x and residual) in flight per thread;
  // few rows: one piece a thread, for the shortest way through the row.  In us, bf16 with a residual, one
  // piece and four: 64 x 4096 2.0 and 2.8, 512 x 4096 3.2 and 4.9, 1024 x 4096 4.9 and 5.2, 4096 x 4096
  // 21.8 and 20.3, 16384 x 512 18.0 and 9.9, 16384 x 8192 168 and 157 (1024 x 2048 goes against it: 3.1 and 4.9).
  if (n > 2048 || (a.T > 512 && n > 32)) return launch_rows<T, 4>(a, st);
  if (n > 1024) return launch_rows<T, 2>(a, st);
  return launch_rows<T, 1>(a, st);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, cudaStream_t st) {
  return dtype == DSV4_BF16 ? launch_type<__nv_bfloat16>(a, st) : launch_type<float>(a, st);
}

}  // namespace dsv4
