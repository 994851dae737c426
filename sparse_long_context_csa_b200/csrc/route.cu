// Routing of tokens to experts: scores from router logits, the choice of topk experts by
// score + bias within the best groups, and the chosen experts' weights.
//
// The order of the choice is that of exact arithmetic.  A warp takes a token and chooses in 32
// bits: every lane sorts the values of its few experts, then the largest head of the warp's lists
// is taken topk times.  A value's last bits make room for its place in the lane, so that sorting
// moves one word per value.  Where two neighbours of the chosen order (or the last group that stays
// and the first that does not) are closer than what is left and fp32's rounding can tell apart,
// which for random logits happens to about one token in five hundred, the warp does the token
// again in 64 bits.  Bound by instruction issue.
#include "common.cuh"
#include "launch.cuh"
#include "moe.h"

namespace dsv4 {
namespace {

// Small CTAs, of which an SM holds as many as the registers allow: for 8 experts a lane 20 warps of
// 96 registers (16384 tokens, 256 experts in 8 groups: 17.6 us; CTAs of 8 warps, 24 warps of 80
// registers, some spilled: 18.9 us; 16 warps: 18.9 us).
constexpr int kWarps = 2;
// CTAs of a kernel with kN experts a lane that an SM holds at once (its registers).  16384 tokens, sigmoid, bias,
// top-8, in us with this many, with fewer and with more: 128 experts 10.3, 12.5 (8 CTAs), 12.0 (16); 256 12.9,
// 13.7 (8), 13.3 (12); 512 32.4, 34.7 (6), 37.1 (10); 1000 89, 115 (3), 93 (6).
constexpr int ctas_of(int kN) { return kN <= 4 ? 12 : kN == 8 ? 10 : kN == 16 ? 8 : 4; }
constexpr unsigned kAll = 0xffffffffu;

// Doubles of shared memory per warp: a value per expert, or 32 integers.
__host__ __device__ constexpr int scratch_of(int E) { return E < 16 ? 16 : E; }
// Words of shared memory per warp for the lanes' sorted lists, without their first two values and
// with three zeros behind the last.  A list that loses its first value then moves one word instead
// of all (16384 tokens, 256 experts in 8 groups: 17.1 us, 17.6 in registers; 512: 36.4 and 42.9; of
// four values a lane no faster).
constexpr int kListed = 8;  // from this many values on
__host__ __device__ constexpr int list_of(int kN) { return kN < kListed ? 0 : 32 * (kN + 1); }

// ---------------------------------------------------------------- 64 bits

// A score is 0 in 64 bits where the logit is below max - 745 (softmax) or -745.
__device__ __forceinline__ double score64(int fn, double l, double mx, double sum) {
  if (fn == DSV4_SCORE_SOFTMAX) return mx == -INFINITY ? 0.0 : exp(l - mx) / sum;
  if (fn == DSV4_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
  return sqrt(log1p(exp(-fabs(l))) + fmax(l, 0.0));
}

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// The largest logit of a row without one above -inf: -inf, or NaN where it holds one (maxima pass over a
// NaN; in other rows the softmax's sum shows it).
template <typename T>
__device__ __noinline__ float largest_of_none(const T* row, int E) {
  bool nan = false;
  for (int e = threadIdx.x & 31; e < E; e += 32) {
    const float l = to_f32<T>(row[e]);
    nan |= l != l;
  }
  return __any_sync(kAll, nan) ? __int_as_float(0x7fffffff) : -INFINITY;
}

// The larger value of the warp, the lower index among equals; index kNone: no value.
constexpr int kNone = 1 << 30;
__device__ __forceinline__ void warp_best(double& v, int& at) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double v2 = __shfl_xor_sync(kAll, v, o);
    const int at2 = __shfl_xor_sync(kAll, at, o);
    if (at2 != kNone && (at == kNone || v2 > v || (v2 == v && at2 < at))) {
      v = v2;
      at = at2;
    }
  }
}

// The chosen experts of one token, lane j the j-th (any E, groups and types); `choice`: E doubles.
template <typename T>
__device__ __noinline__ int choose64(const RouteArgs& a, const T* row, double* choice) {
  const int lane = threadIdx.x & 31;
  double mx = -INFINITY, sum = 0.0;
  if (a.score_fn == DSV4_SCORE_SOFTMAX) {
    for (int e = lane; e < a.E; e += 32) mx = fmax(mx, (double)to_f32<T>(row[e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmax(mx, __shfl_xor_sync(kAll, mx, o));
    if (mx == -INFINITY) mx = (double)largest_of_none<T>(row, a.E);
    for (int e = lane; e < a.E; e += 32) sum += exp((double)to_f32<T>(row[e]) - mx);
    sum = warp_sum64(sum);
  }
  __syncwarp();
  // without a bias the logit chooses, of which every score is a growing function
  const bool lost = sum != sum && mx != -INFINITY;  // a softmax of a NaN or of +inf: every score is NaN
  const double floor_l = a.score_fn == DSV4_SCORE_SOFTMAX ? mx - 745.0 : -745.0;
  for (int e = lane; e < a.E; e += 32) {
    const double l = (double)to_f32<T>(row[e]);
    double c = l < floor_l ? -INFINITY : l;
    if (a.bias) c = score64(a.score_fn, l, mx, sum) + (double)a.bias[e];
    choice[e] = c == c && !lost ? c : -INFINITY;
  }
  __syncwarp();
  if (a.n_group > 1) {
    const int per = a.E / a.n_group;
    double best = -INFINITY;
    if (lane < a.n_group) {
      double b0 = -INFINITY, b1 = -INFINITY;
      for (int i = 0; i < per; ++i) {
        const double c = choice[lane * per + i];
        b1 = c > b0 ? b0 : c > b1 ? c : b1;
        b0 = c > b0 ? c : b0;
      }
      if (!a.bias) {
        b0 = score64(a.score_fn, b0, mx, sum);
        b1 = score64(a.score_fn, b1, mx, sum);
      }
      best = per > 1 ? b0 + b1 : b0;
      if (best != best) best = -INFINITY;
    }
    bool kept = false;
    for (int j = 0; j < a.topk_group; ++j) {
      double v = best;
      int at = lane < a.n_group && !kept ? lane : kNone;
      warp_best(v, at);
      kept |= at == lane;
    }
    const unsigned kept_mask = __ballot_sync(kAll, kept);
    for (int e = lane; e < a.E; e += 32)
      if (!((kept_mask >> (e / per)) & 1u)) choice[e] = nan("");  // not to be chosen
    __syncwarp();
  }
  int mine = 0;
  for (int j = 0; j < a.topk; ++j) {
    double v = 0.0;
    int at = kNone;
    for (int e = lane; e < a.E; e += 32) {
      const double c = choice[e];
      if (c == c && (at == kNone || c > v)) {
        v = c;
        at = e;
      }
    }
    warp_best(v, at);
    if (lane == j) mine = at;
    __syncwarp();
    if (lane == 0) choice[at] = nan("");
    __syncwarp();
  }
  return mine;
}

// The same among `n` <= 31 experts, lane j's e; `at`: 32 integers.
template <typename T>
__device__ __noinline__ int choose_of(const RouteArgs& a, const T* row, int e, int n, double mx, int* at) {
  const int lane = threadIdx.x & 31;
  double sum = 1.0;
  if (a.score_fn == DSV4_SCORE_SOFTMAX && a.bias) {
    sum = 0.0;
    for (int i = lane; i < a.E; i += 32) sum += exp((double)to_f32<T>(row[i]) - mx);
    sum = warp_sum64(sum);
  }
  double c = (double)to_f32<T>(row[e]);
  if (a.bias)
    c = score64(a.score_fn, c, mx, sum) + (double)a.bias[e];
  else if (c < (a.score_fn == DSV4_SCORE_SOFTMAX ? mx - 745.0 : -745.0))
    c = -INFINITY;
  if (!(c == c)) c = -INFINITY;
  int rank = 0;  // of lane's expert
  for (int j = 0; j < n; ++j) {
    const double v = __shfl_sync(kAll, c, j);
    const int f = __shfl_sync(kAll, e, j);
    rank += v > c || (v == c && f < e);
  }
  __syncwarp();
  if (lane < n) at[rank] = e;
  __syncwarp();
  const int mine = lane < n ? at[lane] : 0;
  __syncwarp();
  return mine;
}

// ---------------------------------------------------------------- 32 bits

// Floats as integers in the same order; the lowest is that of -inf, above 0 for every value.
__device__ __forceinline__ uint32_t order_of(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }

// exp(x) and 1 / x to 2 units in the last place, and to 0 where fp32's normal numbers end.
__device__ __forceinline__ float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// fn: known at compile time where it matters.
__device__ __forceinline__ float score32(int fn, float l, float mx, float inv_sum) {
  if (fn == DSV4_SCORE_SIGMOID) return rcp_fast(1.f + exp_fast(-l));
  if (fn == DSV4_SCORE_SOFTMAX) return mx == -INFINITY ? 0.f : exp_fast(l - mx) * inv_sum;
  // e^(l/2), not its square, decides where fp32 ends: below -17 it is the score itself, as
  // log(1 + e) = e (1 - e / 2 + ..) there, which is 1e-8 of it off at most
  const float root = exp_fast(-0.5f * fabsf(l));
  if (l < -17.f) return root;
  // log(1 + e) = 2 atanh(z), z = e / (2 + e) <= 1/3; the terms left out are below 2e-8 of the sum
  const float e = root * root, z = e * rcp_fast(2.f + e), q = z * z;
  float s = fmaf(q, 1.f / 13.f, 1.f / 11.f);
  s = fmaf(q, s, 1.f / 9.f);
  s = fmaf(q, s, 1.f / 7.f);
  s = fmaf(q, s, 1.f / 5.f);
  s = fmaf(q, s, 1.f / 3.f);
  s = fmaf(q * z, s, z);
  return __fsqrt_rn(fmaf(2.f, s, fmaxf(l, 0.f)));
}

// Sorted in descending order (Batcher's odd-even merge sort, kN a power of two).
template <int kN>
__device__ __forceinline__ void sort_down(uint32_t (&k)[kN]) {
#pragma unroll
  for (int p = 1; p < kN; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < kN; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < kN && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t x = k[i + j], y = k[i + j + q];
            k[i + j] = max(x, y);
            k[i + j + q] = min(x, y);
          }
}

// The groups that stay, as a mask, in 64 bits; the layout of route_kernel.  `places`: those of this
// lane's experts e0 + (place << shift) that may be among the two best of their group.
template <typename T>
__device__ __noinline__ unsigned groups_of(const RouteArgs& a, const T* row, int log_lanes, int e0, int shift, uint32_t places,
                                           double mx) {
  const int lane = threadIdx.x & 31, lanes = 1 << log_lanes, per = a.E / a.n_group, g = lane >> log_lanes;
  double sum = 1.0;
  if (a.score_fn == DSV4_SCORE_SOFTMAX) {
    sum = 0.0;
    for (int e = lane; e < a.E; e += 32) sum += exp((double)to_f32<T>(row[e]) - mx);
    sum = warp_sum64(sum);
  }
  double b0 = -INFINITY, b1 = -INFINITY;
  for (; places; places &= places - 1) {
    const int e = e0 + ((__ffs(places) - 1) << shift);
    double c = score64(a.score_fn, (double)to_f32<T>(row[e]), mx, sum) + (a.bias ? (double)a.bias[e] : 0.0);
    c = c == c ? c : -INFINITY;
    b1 = fmax(b1, fmin(b0, c));
    b0 = fmax(b0, c);
  }
  __syncwarp();
  for (int o = 1; o < lanes; o <<= 1) {
    const double m0 = __shfl_xor_sync(kAll, b0, o), m1 = __shfl_xor_sync(kAll, b1, o);
    b1 = fmax(fmin(b0, m0), fmax(b1, m1));
    b0 = fmax(b0, m0);
  }
  double best = per > 1 ? b0 + b1 : b0;
  if (best != best) best = -INFINITY;
  unsigned kept = 0;
  for (int j = 0; j < a.topk_group; ++j) {
    double v = best;
    int at = g < a.n_group && !((kept >> g) & 1u) ? g : kNone;
    warp_best(v, at);
    kept |= 1u << at;
  }
  return kept;
}

// The kN logits from p on, in pieces of up to 16 bytes.
template <typename T, int kN>
__device__ __forceinline__ void load_row(const T* p, float (&l)[kN]) {
  constexpr int kBytes = kN * sizeof(T) < 16 ? kN * sizeof(T) : 16, kPer = kBytes / sizeof(T);
  struct alignas(kBytes) Pack {
    T v[kPer];
  };
#pragma unroll
  for (int j = 0; j < kN; j += kPer) {
    const Pack v = *reinterpret_cast<const Pack*>(p + j);
#pragma unroll
    for (int i = 0; i < kPer; ++i) l[j + i] = to_f32<T>(v.v[i]);
  }
}

// A token per warp at a time.  Group g has the kN * lanes slots of `lanes` = 32 / (n_group rounded
// up to a power of two) neighbouring lanes, its expert j * lanes + i is lane i's j-th.
// kFull: every lane has kN experts, which then are neighbours.
template <typename T, int kN, bool kFull, int fn>
__global__ void __launch_bounds__(kWarps * 32, ctas_of(kN)) route_kernel(RouteArgs a, int log_lanes, int index_bits) {
  extern __shared__ double smem[];
  constexpr int kPlace = kN == 1 ? 0 : kN == 2 ? 1 : kN == 4 ? 2 : kN == 8 ? 3 : kN == 16 ? 4 : 5;
  constexpr float kU = 5.9604645e-8f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lanes = 1 << log_lanes, per = a.E / a.n_group, g = lane >> log_lanes, i = lane & (lanes - 1);
  const int count = g < a.n_group ? (per - i + lanes - 1) >> log_lanes : 0;  // this lane's experts: e0 + (j << shift)
  const int e0 = kFull ? lane * kN : g * per + i, shift = kFull ? 0 : log_lanes;
  // 16-bit logits without a bias are whole in a key's upper half, and the expert's index in the
  // lower one puts equal ones in order; otherwise a key gives up the bits of the place in the lane.
  // The lower half of a 16-bit value's key is zeros, of one below zero ones, which is what the index
  // took the place of: `value` gives the logit itself, where otherwise it gives the lowest value with
  // these upper bits.
  const bool whole = !a.bias && sizeof(T) == 2;
  const int bits = whole ? index_bits : kPlace;
  const uint32_t low = (1u << bits) - 1, lowest = order_of(-INFINITY) & ~low;
  auto value = [&](uint32_t k) {
    if ((k & ~low) == lowest) return -INFINITY;
    return value_of(whole && k < 0x80000000u ? k | low : k & ~low);
  };
  const float cut = __int_as_float((127 + bits - 23) << 23);  // what a key leaves out, of the value

  const uint32_t self = 1u << lane, upto = self | (self - 1);
  double* scratch = smem + (size_t)warp * scratch_of(a.E);
  uint32_t* list = reinterpret_cast<uint32_t*>(smem + (size_t)kWarps * scratch_of(a.E)) + warp * list_of(kN) + lane;
  if constexpr (kN >= kListed) {
#pragma unroll
    for (int j = kN - 2; j < kN + 1; ++j) list[32 * j] = 0u;
  }
  wait_for_previous();
  int64_t t = (int64_t)blockIdx.x * kWarps + warp;
  float bias[kN], most_bias = 0.f;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    bias[j] = a.bias && (kFull || j < count) ? a.bias[e0 + (j << shift)] : 0.f;
    if (fabsf(bias[j]) < INFINITY) most_bias = fmaxf(most_bias, fabsf(bias[j]));
  }
  if (a.bias) most_bias = warp_max(most_bias);
  float l[kN];
  auto load = [&](int64_t token) {
    const T* p = static_cast<const T*>(a.logits) + token * a.E + e0;
    if constexpr (kFull) {
      load_row<T, kN>(p, l);
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j, p += lanes) l[j] = j < count ? to_f32<T>(*p) : -INFINITY;
    }
  };
  if (t < a.T) load(t);
  for (; t < a.T; t += (int64_t)gridDim.x * kWarps) {
    float mx = 0.f, sum = 1.f, inv_sum = 1.f;
    if (fn == DSV4_SCORE_SOFTMAX) {
      mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < kN; ++j) mx = fmaxf(mx, l[j]);
      mx = warp_max(mx);
      if (mx == -INFINITY) mx = largest_of_none<T>(static_cast<const T*>(a.logits) + t * a.E, a.E);
      sum = 0.f;
#pragma unroll
      for (int j = 0; j < kN; ++j) sum += kFull || j < count ? exp_fast(l[j] - mx) : 0.f;
      sum = warp_sum(sum);
      inv_sum = 1.f / sum;
    }
    const bool lost = fn == DSV4_SCORE_SOFTMAX && sum != sum && mx != -INFINITY;  // every score is NaN
    // What is chosen by: score + bias; without a bias the logit, of which every score is a growing
    // function (all that have a score of 0 in 64 bits are as -inf).
    if (a.bias) {
#pragma unroll
      for (int j = 0; j < kN; ++j) l[j] = score32(fn, l[j], mx, inv_sum) + bias[j];
    } else {
      const float floor_l = fn == DSV4_SCORE_SOFTMAX ? mx - 745.f : -745.f;
#pragma unroll
      for (int j = 0; j < kN; ++j) l[j] = l[j] < floor_l ? -INFINITY : l[j] + 0.f;  // -0 is 0
    }
    if (lost) {
#pragma unroll
      for (int j = 0; j < kN; ++j) l[j] = -INFINITY;
    }
    uint32_t key[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const uint32_t place = whole ? low - (uint32_t)(e0 + (j << shift)) : (uint32_t)j;
      key[j] = (order_of(fmaxf(l[j], -INFINITY)) & ~low) | place;  // a NaN is -inf
      if (!kFull && j >= count) key[j] = 0u;
    }
    const int64_t now = t;
    if (t + (int64_t)gridDim.x * kWarps < a.T) load(t + (int64_t)gridDim.x * kWarps);  // the next token's
    sort_down<kN>(key);
    // fp32's rounding, in u = 2^-24, with m the largest score + |bias|: a score s has |ln s| u of itself
    // from exp's argument (the softmax's twice that), which for m above e^-7 stays below 8 m u, and 7 u
    // of itself from exp, the sum and the reciprocal; its sum with the bias is within one more.  The
    // softmax's sum over up to 32 values a lane and 5 steps, of such terms, brings 60 u.  Where all
    // scores are small, |ln s| goes up to 88 before s ends.  Without a bias the logits themselves are
    // compared.
    float blur = 0.f;
    if (a.bias) {
      const float top = value(__reduce_max_sync(kAll, key[0]));
      const float m = fabsf(top) + most_bias;
      blur = (fn == DSV4_SCORE_SOFTMAX ? (m > 1e-3f ? 96.f : 256.f) : m > 1e-3f ? 16.f : 128.f) * kU * m;
    }
    const T* row = static_cast<const T*>(a.logits) + now * a.E;

    if (a.n_group > a.topk_group) {
      // the groups' two best, over the group's lanes
      uint32_t k0 = key[0], k1 = kN > 1 ? key[kN > 1 ? 1 : 0] : 0u;
      for (int o = 1; o < lanes; o <<= 1) {
        const uint32_t m0 = __shfl_xor_sync(kAll, k0, o), m1 = __shfl_xor_sync(kAll, k1, o);
        k1 = max(min(k0, m0), max(k1, m1));
        k0 = max(k0, m0);
      }
      float v0 = value(k0), v1 = per > 1 ? value(k1) : 0.f;
      const float second = per > 1 ? v1 : v0;
      float off = whole ? 0.f : (fabsf(v0) + fabsf(v1)) * cut;  // the bits that the keys left out
      if (a.bias) {
        off += 2.f * blur + 2.f * kU * (fabsf(v0) + fabsf(v1));
      } else {  // scores grow by less than the logit does, the softmax's in proportion to itself
        const float x = fminf(fabsf((fn == DSV4_SCORE_SOFTMAX ? mx : 0.f) - (per > 1 ? v1 : v0)), 90.f);
        v0 = score32(fn, v0, mx, inv_sum);
        v1 = per > 1 ? score32(fn, v1, mx, inv_sum) : 0.f;
        if (fn == DSV4_SCORE_SOFTMAX) off *= v0 + v1;
        off += (2.f * x + 10.f) * kU * (v0 + v1);  // its sum belongs to all of them
      }
      float best = v0 + v1;
      if (!(best == best)) best = -INFINITY;
      const float worst_off = __uint_as_float(__reduce_max_sync(kAll, off < INFINITY ? __float_as_uint(off) : 0u));
      const uint32_t which = 31u >> log_lanes;  // the bits of a group's number
      uint32_t gk = g < a.n_group && i == 0 ? (order_of(best + 0.f) & ~which) | (which - (uint32_t)g) : 0u;
      unsigned kept = 0;
      uint32_t last = 0;
      for (int j = 0; j < a.topk_group; ++j) {
        last = __reduce_max_sync(kAll, gk);
        if (gk == last) gk = 0u;
        kept |= 1u << (which - (last & which));
      }
      const uint32_t next = __reduce_max_sync(kAll, gk);
      const float vl = value_of(last & ~which), vn = value_of(next & ~which);
      // 2^-23: what the bits of the number left out; an infinite score or bias says nothing about the others
      if (!(vl - vn > 2.f * worst_off + 1.2e-7f * (float)(which + 1) * fabsf(vn) + 1e-37f) || !(blur < INFINITY)) {
        uint32_t places = 0;
#pragma unroll
        for (int j = 0; j < kN; ++j)
          if (key[j] != 0u && !(value(key[j]) + fabsf(value(key[j])) * cut + 1e-37f < second - 2.f * blur))
            places |= 1u << (whole ? ((int)(low - (key[j] & low)) - e0) >> shift : (int)(key[j] & low));
        kept = groups_of<T>(a, row, log_lanes, e0, shift, places, (double)mx);
      }
      if (!((kept >> g) & 1u)) {
#pragma unroll
        for (int j = 0; j < kN; ++j) key[j] = 0u;
      }
    }

    // lane j keeps the j-th key and its expert; the one behind the last shows how sure that is
    uint32_t mine_key = 0u, behind = 0u, owners = 0u;
    const uint32_t* rest = list;
    if constexpr (kN >= kListed) {
#pragma unroll
      for (int j = 2; j < kN; ++j) list[32 * (j - 2)] = key[j];
    }
    auto take = [&](int j) {
      const uint32_t best = __reduce_max_sync(kAll, key[0]);
      const uint32_t equal = __ballot_sync(kAll, key[0] == best);  // the lowest lane's is taken
      if (lane == j) {
        mine_key = best;
        owners = equal;
      }
      if ((equal & upto) == self) {
        if constexpr (kN >= kListed) {
          key[0] = key[1];
          key[1] = *rest;
          rest += 32;
        } else {
#pragma unroll
          for (int v = 0; v + 1 < kN; ++v) key[v] = key[v + 1];
          key[kN - 1] = 0u;
        }
      }
      return best;
    };
    for (int j = 0; j <= a.topk; ++j) behind = take(j);
    auto expert = [&]() {
      const int owner = __ffs(owners) - 1;
      const int from = kFull ? owner * kN : (owner >> log_lanes) * per + (owner & (lanes - 1));
      return whole ? (int)(low - (mine_key & low)) : from + ((int)(mine_key & low) << shift);
    };
    int mine = 0;
    bool doubt = false;
    if (!whole) {
      const uint32_t after = __shfl_down_sync(kAll, mine_key, 1), next_key = lane == a.topk - 1 ? behind : after;
      if (lane < a.topk && next_key != 0u) {
        const float vp = value(mine_key), vb = value(next_key);
        doubt = !(vp - vb > fabsf(vb) * cut + 2.f * blur + 1e-37f);
      }
      doubt = __any_sync(kAll, doubt);
    }
    if (!doubt) {
      mine = lane < a.topk ? expert() : 0;
    } else {
      // the order once more in 64 bits, of those that may belong to it: one per lane
      int n = min(a.topk, 32);
      const float last = value(__shfl_sync(kAll, mine_key, a.topk - 1)) - 2.f * blur;
      auto may = [&](uint32_t k) { return k != 0u && !(value(k) + fabsf(value(k)) * cut + 1e-37f < last); };
      uint32_t k = behind;
      while (n < 32 && may(k)) k = take(++n);
      // (lane n's key is the first that does not belong)
      if (lost || n == 32) {
        mine = choose64<T>(a, row, scratch);
      } else {
        mine = choose_of<T>(a, row, lane < n ? expert() : 0, n, (double)mx, reinterpret_cast<int*>(scratch));
      }
    }
    float s = 0.f;
    if (lane < a.topk) s = score32(fn, to_f32<T>(row[mine]), mx, inv_sum);
    if (a.renorm) {
      const float total = warp_sum(s);
      s = __fdividef(s, total + 1e-20f);
    }
    if (lane < a.topk) {
      a.ids[now * a.topk + lane] = mine;
      a.weights[now * a.topk + lane] = s * a.routed_scale;
    }
  }
}

// More experts in a group than 32 registers of its lanes hold: everything in 64 bits.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) route_wide_kernel(RouteArgs a) {
  extern __shared__ double smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
  wait_for_previous();
  if (t >= a.T) return;
  const T* row = static_cast<const T*>(a.logits) + t * a.E;
  const int mine = choose64<T>(a, row, smem + (size_t)warp * scratch_of(a.E));
  float mx = -INFINITY, sum = 0.f;
  if (a.score_fn == DSV4_SCORE_SOFTMAX) {
    for (int e = lane; e < a.E; e += 32) mx = fmaxf(mx, to_f32<T>(row[e]));
    mx = warp_max(mx);
    if (mx == -INFINITY) mx = largest_of_none<T>(row, a.E);
    for (int e = lane; e < a.E; e += 32) sum += exp_fast(to_f32<T>(row[e]) - mx);
    sum = warp_sum(sum);
  }
  float s = 0.f;
  if (lane < a.topk) s = score32(a.score_fn, to_f32<T>(row[mine]), mx, 1.f / sum);
  const float total = warp_sum(s);
  if (lane < a.topk) {
    a.ids[t * a.topk + lane] = mine;
    a.weights[t * a.topk + lane] = (a.renorm ? s / (total + 1e-20f) : s) * a.routed_scale;
  }
}

using RouteKernel = void (*)(RouteArgs, int, int);
template <typename T, int kN, bool kFull>
RouteKernel pick_fn(int fn) {
  return fn == DSV4_SCORE_SOFTMAX ? route_kernel<T, kN, kFull, DSV4_SCORE_SOFTMAX>
         : fn == DSV4_SCORE_SIGMOID ? route_kernel<T, kN, kFull, DSV4_SCORE_SIGMOID>
                                    : route_kernel<T, kN, kFull, DSV4_SCORE_SQRT_SOFTPLUS>;
}
// Full lanes are worth a kernel of their own (fewer tests) from 128 experts on.
template <typename T, int kN>
RouteKernel pick(const RouteArgs& a) {
  constexpr bool kOwn = kN == 4 || kN == 8 || kN == 16;
  return kOwn && a.E == 32 * kN && (a.n_group & (a.n_group - 1)) == 0 ? pick_fn<T, kN, kOwn>(a.score_fn) : pick_fn<T, kN, false>(a.score_fn);
}

template <typename T>
cudaError_t launch_type(const RouteArgs& a, cudaStream_t st) {
  int log_lanes = 5, bits = 0;
  while ((32 >> log_lanes) < a.n_group) --log_lanes;
  while ((1 << bits) < a.E) ++bits;
  const int need = (a.E / a.n_group + (1 << log_lanes) - 1) >> log_lanes;  // experts of a lane
  const int64_t blocks = ((int64_t)a.T + kWarps - 1) / kWarps;
  const int kn = need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : need <= 8 ? 8 : need <= 16 ? 16 : 32;
  const size_t smem = (size_t)kWarps * (scratch_of(a.E) * sizeof(double) + list_of(kn) * sizeof(uint32_t));
  const auto fn = need <= 1 ? pick<T, 1>(a) : need <= 2 ? pick<T, 2>(a) : need <= 4 ? pick<T, 4>(a) : need <= 8 ? pick<T, 8>(a) :
                  need <= 16 ? pick<T, 16>(a) : pick<T, 32>(a);
  static_assert(kWarps * (kMaxExperts * sizeof(double) + list_of(32) * sizeof(uint32_t)) <= 48 * 1024, "");
  if (need > 32) return launch(route_wide_kernel<T>, blocks, kWarps * 32, smem, st, a);
  const int64_t held = (int64_t)sm_count() * ctas_of(kn);
  return launch(fn, blocks < held ? blocks : held, kWarps * 32, smem, st, a, log_lanes, bits);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, int dtype, cudaStream_t st) {
  return dtype == DSV4_BF16 ? launch_type<__nv_bfloat16>(a, st) : launch_type<float>(a, st);
}

}  // namespace dsv4
