// The experts' products of a routed layer:
//   out[t] = sum_j weights[t,j] * W2_e h,  h = silu(g) * u,  g = W1_e x_t,  u = W3_e x_t,  e = ids[t,j]
// with g <- min(g, limit) and u <- clamp(u, -limit, limit) when a limit is given.
// The (token, choice) pairs are put in order of their expert; h is rounded to bf16 (the type of
// the second product's operands; with few tokens, on the CUDA cores, it stays in 32 bits), the
// products of a pair are kept in 32 bits until the sum over j.
#include <cuda.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"
#include "launch.cuh"
#include "moe.h"
#include "tc_pair.cuh"

namespace dsv4 {

__device__ int g_experts_error = 0;

namespace {

// Chunks that the pairs are counted and placed in: one CTA each.
constexpr int kMaxChunks = 64, kOrderThreads = 1024;
constexpr int64_t kOneCta = 4096;  // pairs that a single CTA orders
constexpr int kFewPairs = 32;      // pairs that the few-token path takes
// Pairs that the gather puts in order by itself, one launch less (4 tokens, 2 of 8 experts of 1024 x
// 512: 18.1 us, 19.4 with a kernel for the order; 384 pairs of 64: 54.6 and 55.6; 1020 pairs no faster,
// 4096 pairs 4 us slower).
constexpr int64_t kPlaced = 512;

struct Layout {
  size_t offs, slot_row, counts, h, yp, total;
};
Layout layout(int64_t T, int hidden, int inter, int E, int topk) {
  const int64_t n = T * topk;
  Layout l{};
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  l.offs = 0;
  l.slot_row = up((size_t)(E + 1) * 4);
  l.counts = l.slot_row + up((size_t)n * 4);
  l.h = l.counts + (n > kOneCta ? up((size_t)kMaxChunks * E * 4) : 0);
  // bf16, or of up to kFewPairs pairs fp32; every part grows with every size, so that the workspace of a
  // larger call serves a smaller one
  const size_t few = (size_t)(n < kFewPairs ? n : kFewPairs) * 4, all = (size_t)n * 2;
  l.yp = l.h + up((few > all ? few : all) * inter);
  l.total = l.yp + up((size_t)n * hidden * 4);
  return l;
}

__device__ __forceinline__ bool is_expert(int e, int E) { return e >= 0 && e < E; }

// The sum of the values of the threads before this one; all kOrderThreads threads take part.
__device__ __forceinline__ int exclusive_scan(int v, int* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int w = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    part[lane] = w;
  }
  __syncthreads();
  return s - v + (warp > 0 ? part[warp - 1] : 0);
}

// Pairs of chunk blockIdx.x by expert.
__global__ void __launch_bounds__(kOrderThreads) count_kernel(const int32_t* ids, int64_t n, int64_t chunk, int E,
                                                              int32_t* counts) {
  __shared__ int32_t count[kMaxExperts];
  wait_for_previous();
  for (int e = threadIdx.x; e < E; e += kOrderThreads) count[e] = 0;
  __syncthreads();
  const int64_t end = min(n, (blockIdx.x + 1) * chunk);
  for (int64_t i = blockIdx.x * chunk + threadIdx.x; i < end; i += kOrderThreads)
    if (is_expert(ids[i], E)) atomicAdd(&count[ids[i]], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kOrderThreads) counts[(int64_t)blockIdx.x * E + e] = count[e];
}

// Rows of the pairs in order of their expert.  One CTA counts for itself (counts NULL); of
// several, each takes the chunks before its own from count_kernel.  Which row of its expert a pair
// gets within a chunk is left to the atomics: a row's products do not depend on its place.
__global__ void __launch_bounds__(kOrderThreads) order_kernel(const int32_t* ids, int64_t n, int64_t chunk, int E,
                                                              const int32_t* counts, int32_t* offs, int32_t* slot_row) {
  __shared__ int32_t at[kMaxExperts], part[32];
  wait_for_previous();
  const int e = threadIdx.x;  // E <= kOrderThreads
  int total = 0, before = 0;
  if (counts) {
    if (e < E) {
#pragma unroll 8
      for (int c = 0; c < (int)gridDim.x; ++c) {
        const int v = counts[(int64_t)c * E + e];
        total += v;
        before += c < (int)blockIdx.x ? v : 0;
      }
    }
  } else {
    if (e < E) at[e] = 0;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += kOrderThreads)
      if (is_expert(ids[i], E)) atomicAdd(&at[ids[i]], 1);
    __syncthreads();
    total = e < E ? at[e] : 0;
  }
  const int start = exclusive_scan(total, part);
  if (e < E) {
    at[e] = start + before;
    if (blockIdx.x == 0) {
      offs[e] = start;
      if (e == E - 1) offs[E] = start + total;
    }
  }
  __syncthreads();
  const int64_t end = min(n, (blockIdx.x + 1) * chunk);
  for (int64_t i = blockIdx.x * chunk + threadIdx.x; i < end; i += kOrderThreads) {
    slot_row[i] = is_expert(ids[i], E) ? atomicAdd(&at[ids[i]], 1) : -1;
  }
}

// ---------------------------------------------------------------- the two products
//
// One kernel, a CTA pair per 256 x N tile: D[256 weight rows, N token rows] = W X^T, so that the
// ragged side (the rows of one expert) is N, which an MMA takes in steps of 16, and few rows cost
// little.  Each CTA of the pair holds 128 weight rows and half of the token rows.
//  * warps 0 and 6: TMA producers of the weights and of the token rows, a ring of stages of 64
//    channels (16 KB and up to 16 KB).  One thread's turn costs 200 clocks and 150 per load, and a
//    step of the MMAs takes 512 clocks for 256 rows, 400 for few: so each of the two issues one
//    load a turn, and a stage's barrier is asked for a step ahead.
//  * warp 1 (of the leader): M=256, K=16 MMAs into one of two 256-column accumulators, so that
//    a tile's epilogue overlaps the next tile's main loop.
//  * warps 2-5: epilogue, one TMEM lane quadrant each.
// First product (kPass 0): the TMA box interleaves 16 gate rows with 16 up rows, so that lanes l
// and l + 16 of an epilogue warp hold gate and up of one channel and one shuffle brings both
// together; h goes out in bf16.  Second product: y in fp32, a row of 32 channels per store.
// A tile's rows behind its expert's last one are the next expert's (or the fill's): their columns
// are computed and not stored.  Every wait is bounded; a role that gives up records
// g_experts_error and leaves, and the others time out behind it.
constexpr int kBK = 64, kStages = 7, kMaxN = 256;  // kStages: at most
constexpr uint32_t kStageA = 128 * kBK * 2, kStageB = (kMaxN / 2) * kBK * 2;
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr int kGemmThreads = 224;

struct GemmParams {
  int N;        // output channels (inter, hidden)
  int K;        // reduction length
  int E;
  int rows;     // of `out`, which all offsets are held to
  int stages;   // of the ring
  float limit;
  const int32_t* offs;  // [E+1] first row of each expert
  void* out;    // h (bf16) or y (fp32), [rows, N]
};

// Tensor maps of the token rows in boxes of 16, 32, 64 and 128: a load costs the thread that issues it
// some 150 clocks whatever its size, so that a tile's rows come in one.
constexpr int kRowMaps = 4;
struct RowMaps {
  CUtensorMap box[kRowMaps];
};

struct Bars {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
  uint32_t tmem_base;
};
constexpr uint32_t kSmemMost = 227 * 1024;
// Stages, then the barriers (1 KB), then the experts' offsets.
constexpr uint32_t gemm_smem(int stages, int E) { return stages * (kStageA + kStageB) + 1024 + (E + 1) * 4; }

// Walks the tiles of all experts in order: expert, then weight tile, then row tile.
struct Cursor {
  const int32_t* offs;
  int E, wt;                 // weight tiles of an expert
  int e = 0, n = 0, nt = 0;  // expert, its rows, its row tiles
  int64_t base = 0;          // tiles before expert e
  __device__ Cursor(const int32_t* o, int experts, int weight_tiles) : offs(o), E(experts), wt(weight_tiles) { open(); }
  __device__ void open() {
    n = e < E ? max(offs[e + 1] - offs[e], 0) : 0;
    nt = (n + kMaxN - 1) / kMaxN;
  }
  // Tile t (never below the last one asked for): its weight tile, first row and rows; false: none.
  __device__ bool at(int64_t t, int* w, int* row, int* rows) {
    while (e < E && t >= base + (int64_t)wt * nt) {
      base += (int64_t)wt * nt;
      ++e;
      open();
    }
    if (e >= E) return false;
    const int i = (int)(t - base), k = i % nt;
    const int per = ((n + nt - 1) / nt + 15) / 16 * 16;  // the tiles of an expert are of one height
    *w = i / nt;
    *row = offs[e] + k * per;
    *rows = min(per, n - k * per);
    return true;
  }
};

template <int kPass>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ RowMaps maps,
                const __grid_constant__ GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = tc::cluster_cta_rank();
  const int stages = p.stages;
  Bars* bars = reinterpret_cast<Bars*>(smem + stages * (kStageA + kStageB));
  int32_t* offs = reinterpret_cast<int32_t*>(smem + stages * (kStageA + kStageB) + 1024);
  const int k_steps = (p.K + kBK - 1) / kBK;
  const int weight_tiles = kPass == 0 ? (p.N + 127) / 128 : (p.N + 255) / 256;
  const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
  bool aligned = (tc::smem_u32(smem) & 1023u) == 0;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&bars->full[s], 1);
      tc::mbar_init(&bars->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&bars->acc_full[b], 1);
      tc::mbar_init(&bars->acc_empty[b], 8);  // the epilogue warps of both CTAs
    }
    tc::mbar_fence_init();
  }
  if (warp == 1) {
    tc::tmem2_alloc(&bars->tmem_base, 512);
    tc::tmem2_relinquish();
  }
  wait_for_previous();
  // Whoever writes to the workspace during the call (a second call that was given the same one, a fill
  // on another stream) spoils its results and nothing outside: offsets and rows stay within the workspace.
  for (int e = tid; e <= p.E; e += kGemmThreads) offs[e] = min(max(p.offs[e], 0), p.rows);
  if (tid == 0) {
    tc::prefetch_tensormap(&map_w);
    for (int i = 0; i < kRowMaps; ++i) tc::prefetch_tensormap(&maps.box[i]);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (!aligned) {
    if (tid == 0) atomicExch(&g_experts_error, 3);
  } else if (warp == 0 || warp == 6) {
    // ------------------------------------------------------------------ TMA producers
    if (lane == 0) {
      const bool weights = warp == 0;
      Cursor cur(offs, p.E, weight_tiles);
      int s = 0;
      uint32_t phase = 1;            // the first round finds every stage free
      bool ok = true, free = false;  // free: stage s is known to be
      bool first = true;
      const uint32_t full0 = tc::cluster_addr(&bars->full[0], 0);
      int w, row, rows;
      for (int64_t t = pair; ok && cur.at(t, &w, &row, &rows); t += pairs) {
        const int half = (rows + 15) / 16 * 8;  // token rows of one CTA
        const int y = row + (int)rank * half;
        const int size = half > 64 ? 3 : half > 32 ? 2 : half > 16 ? 1 : 0;  // one box of 16 << size rows
        const CUtensorMap* map = &maps.box[size];
        const uint32_t bytes = 2 * (kStageA + (16u << size) * kBK * 2);
        const int y_w = kPass == 0 ? w * 8 + (int)rank * 4 : w * 256 + (int)rank * 128;
        for (int k = 0; k < k_steps; ++k) {
          if (!free && !first && !tc::mbar_wait(&bars->empty[s], phase, kWaitLimit)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * (kStageA + kStageB);
          uint64_t* here = &bars->full[s];
          const uint32_t full = full0 + s * 8;
          if (++s == stages) {
            s = 0;
            phase ^= 1u;
            first = false;
          }
          if (weights) {
            if (rank == 0) tc::mbar_arrive_expect_tx(here, bytes);
            free = kPass == 0 ? tc::tma2_load_5d_test(sa, &map_w, k * kBK, 0, 0, y_w, cur.e, full, &bars->empty[s], phase)
                              : tc::tma2_load_3d_test(sa, &map_w, k * kBK, y_w, cur.e, full, &bars->empty[s], phase);
          } else {
            free = tc::tma2_load_2d_test(sa + kStageA, map, k * kBK, y, full, &bars->empty[s], phase);
          }
        }
      }
      if (!ok) {
        atomicExch(&g_experts_error, 1);
        // copies in flight: those of this round, and of the one before it (a stage's full phase of a
        // round is the one that `phase` was not)
        for (int i = 0; i < stages && rank == 0; ++i)
          if (i < s || !first) (void)tc::mbar_wait(&bars->full[i], i < s ? phase ^ 1u : phase, kWaitLimit);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (the leader's)
    if (rank == 0 && lane == 0) {
      Cursor cur(offs, p.E, weight_tiles);
      int s = 0;
      uint32_t phase = 0, lt = 0;
      bool ok = true, full = false;  // full: stage s is known to be
      const uint32_t smem0 = tc::smem_u32(smem);
      int w, row, rows;
      for (int64_t t = pair; ok && cur.at(t, &w, &row, &rows); t += pairs, ++lt) {
        const int buf = (int)(lt & 1);
        if (lt >= 2 && !tc::mbar_wait(&bars->acc_empty[buf], ((lt >> 1) - 1) & 1, kWaitLimit)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t idesc = tc::idesc_bf16_f32(256, (rows + 15) / 16 * 16, 0, 0);
        const uint32_t acc = tmem + buf * kMaxN;
        for (int k = 0; k < k_steps; ++k) {
          if (!full && !tc::mbar_wait(&bars->full[s], phase, kWaitLimit)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint32_t a0 = smem0 + s * (kStageA + kStageB);
          uint64_t* done = &bars->empty[s];  // free in both CTAs once these MMAs have read it
          if (++s == stages) {
            s = 0;
            phase ^= 1u;
          }
          full = tc::umma2_f16_step(acc, tc::sdesc_sw128(a0, 16, 1024), tc::sdesc_sw128(a0 + kStageA, 16, 1024), idesc,
                                    k > 0 ? 1u : 0u, done, &bars->full[s], phase);
        }
        if (ok) tc::umma2_commit_both(&bars->acc_full[buf]);
      }
      if (!ok) atomicExch(&g_experts_error, 2);
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q4 = warp & 3;  // TMEM lane quadrant this warp may access
    Cursor cur(offs, p.E, weight_tiles);
    uint32_t lt = 0;
    bool ok = true;
    int w, row, rows;
    for (int64_t t = pair; cur.at(t, &w, &row, &rows); t += pairs, ++lt) {
      const int buf = (int)(lt & 1);
      if (!__all_sync(0xffffffffu, tc::mbar_wait(&bars->acc_full[buf], (lt >> 1) & 1, kWaitLimit))) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      const uint32_t acc = tmem + buf * kMaxN + ((uint32_t)(q4 * 32) << 16);
      if (kPass == 0) {
        const int c = w * 128 + (int)rank * 64 + q4 * 16 + (lane & 15);
        const bool up = lane >= 16;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (int64_t)row * p.N + c;
        for (int j = 0; j < rows; j += 32) {
          float v[32];
          tc::tmem_ld_x32(acc + j, v);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            // lane l keeps column i, lane l + 16 column i + 1
            const float other = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 1], 16);
            float g = up ? other : v[i], u = up ? v[i + 1] : other;
            const int m = j + i + (up ? 1 : 0);
            if (p.limit > 0.f) {
              g = g > p.limit ? p.limit : g;  // a NaN stays one
              u = u > p.limit ? p.limit : u < -p.limit ? -p.limit : u;
            }
            if (m < rows && c < p.N) dst[(int64_t)m * p.N] = __float2bfloat16_rn(__fdividef(g, 1.f + __expf(-g)) * u);
          }
        }
      } else {
        const int c = w * 256 + (int)rank * 128 + q4 * 32 + lane;
        float* dst = static_cast<float*>(p.out) + (int64_t)row * p.N + c;
        for (int j = 0; j < rows; j += 32) {
          float v[32];
          tc::tmem_ld_x32(acc + j, v);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (j + i < rows && c < p.N) dst[(int64_t)(j + i) * p.N] = v[i];
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster(tc::cluster_addr(&bars->acc_empty[buf], 0));
    }
    if (!ok && lane == 0) atomicExch(&g_experts_error, 4);
  }

  __syncwarp();
  tc::tc_fence_before();
  tc::cluster_sync();  // the peer's shared memory and barriers are in use until here
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem2_dealloc(tmem, 512);
  }
}

// Eight e4m3 values and their scale, as the bf16 values that they stand for.
__device__ __forceinline__ uint4 dequantise(uint2 q, float s) {
  uint4 o;
  uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)((j < 2 ? q.x : q.y) >> (16 * (j & 1)));
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return o;
}

// Rows of x in order of their expert, as bf16.  A warp reads a piece of a token's row once, kUnroll
// times 16 bytes per lane, and writes it to all of its places (of 2048 tokens or more), or to one
// (of fewer, for more warps).  Calls of 16-bit rows with all places and with one: 2048 x 2048, 4 choices, 212
// and 204 us; 2048 x 4096 548 and 549; 6000 x 1024, 6 choices, 272 and 320.  In the order of the rows, x is read again
// for every choice once it no longer fits L2 beside what is written (8192 x 4096, 6 choices: 127 us
// instead of 94).
// kPlace (a few pairs): the first E + 1 warps find the experts' first rows, the others their pair's
// row, each by a look at all ids; nothing is put in order before, and splits is topk.
constexpr int kGatherWarps = 8, kUnroll = 8, kPiece = 32 * kUnroll;
template <bool kPlace>
__global__ void __launch_bounds__(kGatherWarps * 32) gather_kernel(ExpertArgs a, int pieces, int splits, int32_t* offs,
                                                                  int32_t* slot_row, __nv_bfloat16* xp) {
  wait_for_previous();
  const int lane = threadIdx.x & 31, per = pieces * splits;
  int64_t unit = (int64_t)blockIdx.x * kGatherWarps + (threadIdx.x >> 5);
  // The pairs of the experts before e, and those of e before pair i.
  auto row_of = [&](int e, int i) {
    const int n = a.T * a.topk;
    int sum = 0;
#pragma unroll 4
    for (int j = lane; j < n; j += 32) {
      const int id = a.ids[j];
      sum += (id >= 0 && id < e) || (id == e && j < i);
    }
    return __reduce_add_sync(0xffffffffu, sum);
  };
  if (kPlace) {
    if (unit <= a.E) {
      const int first = row_of((int)unit, 0);
      if (lane == 0) offs[unit] = first;
      return;
    }
    unit -= a.E + 1;
  }
  const int64_t t = unit / per;
  if (t >= a.T) return;
  const int rest = (int)(unit - t * per), split = rest / pieces, i0 = (rest - split * pieces) * kPiece + lane;
  const int n = a.hidden / 8;
  uint4 v[kUnroll];
  if (a.x_scale) {
    const uint2* src = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + t * a.hidden);
    const float* sc = a.x_scale + t * ((a.hidden + kScaleGroup - 1) / kScaleGroup);
    uint2 q[kUnroll];
    float f[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {  // all loads first
      const int i = min(i0 + 32 * u, n - 1);
      q[u] = src[i];
      f[u] = sc[i / (kScaleGroup / 8)];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = dequantise(q[u], f[u]);
  } else {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + t * a.hidden);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = src[min(i0 + 32 * u, n - 1)];
  }
  for (int j = split; j < a.topk; j += splits) {
    const int64_t i = t * a.topk + j;
    int r;
    if (kPlace) {
      const int e = a.ids[i];
      r = is_expert(e, a.E) ? row_of(e, (int)i) : -1;
      if (lane == 0) slot_row[i] = r;  // every piece's warp the same
    } else {
      r = slot_row[i];
    }
    if ((uint32_t)r >= (uint32_t)(a.T * a.topk)) continue;  // -1: dropped
    uint4* dst = reinterpret_cast<uint4*>(xp + (int64_t)r * a.hidden);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i0 + 32 * u < n) dst[i0 + 32 * u] = v[u];
  }
}

// out[t] = sum_j weights[t,j] y(t,j) in the order of j: a CTA per token and part of its channels,
// four channels a thread at a time, the rows of kJ choices in flight.
constexpr int kJ = 8, kCombineThreads = 256;
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(ExpertArgs a, int parts, const int32_t* slot_row, const float* yp) {
  wait_for_previous();
  const int64_t t = blockIdx.x / parts;
  const int n = a.hidden / 4, part = (int)(blockIdx.x - t * parts);
  const int32_t* places = slot_row + t * a.topk;
  const float* weights = a.weights + t * a.topk;
  uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + t * a.hidden);
#pragma unroll 2
  for (int i = part * kCombineThreads + threadIdx.x; i < n; i += parts * kCombineThreads) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < a.topk; j0 += kJ) {
      float4 v[kJ];
      float w[kJ];
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        w[j] = 0.f;
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j0 + j < a.topk) {
          const int r = places[j0 + j];
          if ((uint32_t)r < (uint32_t)(a.T * a.topk)) {  // -1: dropped
            w[j] = weights[j0 + j];
            v[j] = __ldcs(reinterpret_cast<const float4*>(yp + (int64_t)r * a.hidden) + i);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        s.x += w[j] * v[j].x;
        s.y += w[j] * v[j].y;
        s.z += w[j] * v[j].z;
        s.w += w[j] * v[j].w;
      }
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
    uint2 o;
    o.x = *reinterpret_cast<const uint32_t*>(&lo);
    o.y = *reinterpret_cast<const uint32_t*>(&hi);
    out[i] = o;
  }
}

// ---------------------------------------------------------------- few tokens
//
// With a handful of pairs the weights of the chosen experts are read once and nothing else counts:
// matrix-vector products on the CUDA cores, without ordering, gathering and combining.  One CTA
// per SM takes an even share of the weight rows.  Its producer warp streams them through a ring in
// shared memory with bulk copies.  A stage is about 32 KB: a turn of the ring costs its threads
// some 550 clocks, so that stages of 4, 8, 16 and 32 KB stream 2.1, 4.1, 6.9 and 7.0 TB/s (805 MB,
// nothing else done).  96 KB of ring let the CTAs of both products fit an SM, so that the second
// one fills its ring while the first one ends.  The eight consumer warps divide a row's channels:
// each keeps its part of the tokens' rows in registers and reads nothing but weights, two channels
// a multiply-add.  A warp's part of a dot goes to shared memory; every 32 items the warps meet and
// the parts are summed, always in the same order.  What bounds it is the consumers' latency: one
// token of six experts (4096 x 2048, 302 MB) takes 58 us, 5.2 TB/s (65 us with single multiply-adds,
// 85 us with a meeting at every stage).
// More tokens than three go through the tensor cores: four of six experts take 181 us there and
// 278 us here, where the rows of more than kFewRows pairs of an expert are streamed again.
constexpr int kFewTokens = 3, kFewWarps = 8, kFewRows = 2, kFlush = 32;
constexpr int kFewThreads = (kFewWarps + 1) * 32;
constexpr uint32_t kFewRing = 96 * 1024;
constexpr int kFewStages = 8;    // at most
constexpr int kFewWidth = 8192;  // channels of a row at most

struct FewShared {
  uint64_t full[kFewStages], empty[kFewStages];
  float part[2][kFlush][2 * kFewRows][kFewWarps];  // [item][gate, up][pair][warp of the row]
  float sum[];  // second product: [channels of the CTA][kFewTokens]
};

// The pairs, one per lane (at most 32): which of them share an expert, and the first of each.
struct FewPairs {
  int id;            // this lane's expert, -1: none
  unsigned same;     // lanes with the same one
  unsigned leaders;  // first lanes of the experts that are asked for
  __device__ explicit FewPairs(const ExpertArgs& a) {
    const int lane = threadIdx.x & 31;
    id = lane < a.T * a.topk ? a.ids[lane] : -1;
    if (!is_expert(id, a.E)) id = -1;
    same = __match_any_sync(0xffffffffu, id);
    leaders = __ballot_sync(0xffffffffu, id >= 0 && __ffs(same) - 1 == lane);
  }
};

// How a row's channels and the rows are divided: kP pieces of eight channels per lane, `wide` warps
// per row, `side` rows at a time, `batch` times in a stage.
struct FewShape {
  int wide, side, batch, stages;
  uint32_t row_bytes, stage_bytes;
  __device__ FewShape(int K, int P, int rows_per_item, int items) {
    wide = (K / 8 + 32 * P - 1) / (32 * P);
    side = kFewWarps / wide;
    batch = items;
    row_bytes = (uint32_t)K * 2;
    stage_bytes = (uint32_t)(batch * side * rows_per_item) * row_bytes;
    stages = min((int)(kFewRing / stage_bytes), kFewStages);
  }
};

// Two fp32 values in a register pair, and two fused multiply-adds at once.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float sum_of(uint64_t p) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
  return lo + hi;
}
// Two bf16 values of a word.
__device__ __forceinline__ uint64_t pair_of(uint32_t w) { return pair_of(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   tc::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}

// The sums over the warp of kV (a power of two) values per lane: value i in lanes
// i * (32 / kV) .. of the result, with kV - 1 + log2(32 / kV) shuffles.
template <int kV>
__device__ __forceinline__ float sum_transposed(float (&v)[kV]) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int n = kV / 2; n >= 1; n >>= 1, o >>= 1) {
    const bool hi = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float got = __shfl_xor_sync(0xffffffffu, hi ? v[i] : v[i + n], o);
      v[i] = (hi ? v[i + n] : v[i]) + got;
    }
  }
  float r = v[0];
#pragma unroll
  for (; o >= 1; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  return r;
}

// The i-th set bit of a mask, -1: there are fewer.
__device__ __forceinline__ int nth_bit(unsigned m, int i) {
  for (; i > 0; --i) m &= m - 1;
  return __ffs(m) - 1;
}

// A role's place in the ring.
struct FewWalk {
  int stage = 0;
  uint32_t phase = 0;
  int part = 0;  // which half of FewShared::part is next
  __device__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// Turns of a stage: 32 KB of rows of kP * 2048 channels.
template <bool kUp, int kP>
constexpr int few_batch() { return (kUp ? 4 : 8) / kP; }

// The items of one expert (`count` weight rows from `row0` on) for all of its pairs, by a consumer
// warp; kR of the pairs at a time.
template <bool kUp, int kP, int kR>
__device__ __forceinline__ bool few_expert(const ExpertArgs& a, const FewShape& fs, uint8_t* smem, FewShared* sh, FewWalk& at,
                                           int row0, int count, unsigned mine, float* h, int c0) {
  constexpr int kNR = kUp ? 2 : 1, kBatch = few_batch<kUp, kP>(), kV = kBatch * kNR * kR, kPer = 32 / kV;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  static_assert(kBatch * kFewWarps <= kFlush && kV <= 32 && 2 * kFewRows >= kNR * kR, "a stage's parts fit FewShared::part");
  const int kw = warp % fs.wide, g = warp / fs.wide, workers = fs.wide * fs.side * 32;
  const int K8 = (kUp ? a.hidden : a.inter) / 8, piece = kw * 32 * kP + lane;
  const int step = kBatch * fs.side, rows = __popc(mine);
  // the items between two meetings: whole stages, or one stage where it has more
  const int flush = max(kFlush / step, 1) * step;
  const int value = lane / kPer;  // this lane's of the kV dots: [turn][gate, up][pair]
  const int value_item = value / (kNR * kR) * fs.side + g, value_dot = value % (kNR * kR);
  const uint32_t hop = fs.side * fs.row_bytes;
  const bool whole_part = (kw + 1) * 32 * kP <= K8;  // no lane of the warp is behind the row's end
  for (int first = 0; first < rows; first += kR) {
    // this lane's part of the pairs' rows
    uint64_t x[kR][kP][4];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int slot = max(nth_bit(mine, first + r), 0);
#pragma unroll
      for (int q = 0; q < kP; ++q) {
        const int i = piece + 32 * q;
        if (!kUp) {
          float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
          if (i < K8) {
            const float4* row = reinterpret_cast<const float4*>(h) + ((int64_t)slot * K8 + i) * 2;
            lo = row[0];
            hi = row[1];
          }
          x[r][q][0] = pair_of(lo.x, lo.y);
          x[r][q][1] = pair_of(lo.z, lo.w);
          x[r][q][2] = pair_of(hi.x, hi.y);
          x[r][q][3] = pair_of(hi.z, hi.w);
        } else {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (i < K8) {
            const int64_t t = slot / a.topk;
            if (a.x_scale)
              v = dequantise(static_cast<const uint2*>(a.x)[t * K8 + i],
                             a.x_scale[t * ((a.hidden + kScaleGroup - 1) / kScaleGroup) + i / (kScaleGroup / 8)]);
            else
              v = static_cast<const uint4*>(a.x)[t * K8 + i];
          }
          const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) x[r][q][j] = pair_of(words[j]);
        }
      }
    }
    for (int i0 = 0; i0 < count; i0 += flush) {
      const int n = min(flush, count - i0);
      float (*part)[2 * kFewRows][kFewWarps] = sh->part[at.part];
      bool ok = true;
      for (int i = 0; i < n && ok; i += step) {
        uint64_t acc[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v) acc[v] = 0;
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&sh->full[at.stage], at.phase, kWaitLimit));
        // Rows that a last stage lacks are whatever the ring holds: their dots are not looked at.
        const uint8_t* w0 = smem + at.stage * fs.stage_bytes + g * fs.row_bytes + piece * 16;
        auto dots = [&](auto whole) {
#pragma unroll
          for (int item = 0; item < kNR * kBatch; ++item) {
            const int v = (item % kBatch * kNR + item / kBatch) * kR;  // rows lie by (gate, up), turn
#pragma unroll
            for (int q = 0; q < kP; ++q) {
              if (!whole.value && piece + 32 * q >= K8) continue;
              const uint4 w = *reinterpret_cast<const uint4*>(w0 + item * hop + q * 512);
              const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint64_t two = pair_of(words[j]);
#pragma unroll
                for (int r = 0; r < kR; ++r) acc[v + r] = fma2(two, x[r][q][j], acc[v + r]);
              }
            }
          }
        };
        if (whole_part)
          dots(std::true_type{});
        else
          dots(std::false_type{});
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh->empty[at.stage]);
        at.next(fs.stages);
        float sums[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v) sums[v] = sum_of(acc[v]);
        const float dot = sum_transposed<kV>(sums);
        if (lane % kPer == 0) part[i + value_item][value_dot][kw] = dot;
      }
      at.part ^= 1;
      if (!tc::named_bar_and(1, workers, ok)) return false;
      // a thread per item; the next write to this half of the parts is behind the next meeting
      for (int i = warp * 32 + lane; i < n; i += workers) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const int slot = nth_bit(mine, first + r);
          if (slot < 0) break;
          float d[kNR];
#pragma unroll
          for (int nr = 0; nr < kNR; ++nr) {
            d[nr] = 0.f;
            for (int w = 0; w < fs.wide; ++w) d[nr] += part[i][nr * kR + r][w];
          }
          if (kUp) {
            float gate = d[0], u = d[kNR - 1];
            if (a.limit > 0.f) {
              gate = gate > a.limit ? a.limit : gate;  // a NaN stays one
              u = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
            }
            h[(int64_t)slot * a.inter + row0 + i0 + i] = __fdividef(gate, 1.f + __expf(-gate)) * u;
          } else {
            sh->sum[(row0 + i0 + i - c0) * kFewTokens + slot / a.topk] += a.weights[slot] * d[0];
          }
        }
      }
    }
  }
  return true;
}

template <bool kUp, int kP>
__global__ void __launch_bounds__(kFewThreads, 2) few_kernel(ExpertArgs a, float* h) {
  constexpr int kNR = kUp ? 2 : 1, kBatch = few_batch<kUp, kP>();
  extern __shared__ __align__(1024) uint8_t smem[];
  FewShared* sh = reinterpret_cast<FewShared*>(smem + kFewRing);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const FewShape fs(kUp ? a.hidden : a.inter, kP, kNR, kBatch);
  // this CTA's share: of the (expert, channel) units in order; of the output channels
  const int c0 = (int)((int64_t)a.hidden * blockIdx.x / gridDim.x), c1 = (int)((int64_t)a.hidden * (blockIdx.x + 1) / gridDim.x);
  if (threadIdx.x < fs.stages) {
    tc::mbar_init(&sh->full[threadIdx.x], 1);
    tc::mbar_init(&sh->empty[threadIdx.x], fs.wide * fs.side);
  }
  if (!kUp)
    for (int i = threadIdx.x; i < (c1 - c0) * kFewTokens; i += kFewThreads) sh->sum[i] = 0.f;
  tc::mbar_fence_init();
  __syncthreads();
  // The first product waits for what is before the call and only then lets the second one start,
  // which therefore finds ids, weights and x as they are to be and waits for h alone.
  if (kUp) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const FewPairs pairs(a);
  const int64_t units = (int64_t)__popc(pairs.leaders) * a.inter;
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  const bool producer = warp == kFewWarps;
  if (!kUp && !producer) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (producer || warp < fs.wide * fs.side) {
    int64_t base = 0;  // units before the expert
    FewWalk at;
    int rounds = 0;    // of the ring, by the producer
    bool ok = true;
    for (unsigned left = pairs.leaders; left && ok; left &= left - 1, base += a.inter) {
      const int leader = __ffs(left) - 1;
      const int row0 = kUp ? (int)max(u0 - base, (int64_t)0) : c0;
      const int row1 = kUp ? (int)min(u1 - base, (int64_t)a.inter) : c1;
      const int count = row1 - row0;
      if (count <= 0) continue;
      const int64_t e = __shfl_sync(0xffffffffu, pairs.id, leader);
      const unsigned mine = __shfl_sync(0xffffffffu, pairs.same, leader);
      if (producer) {
        if (lane == 0) {
          const __nv_bfloat16* w = kUp ? static_cast<const __nv_bfloat16*>(a.w13) + (e * 2 * a.inter + row0) * a.hidden
                                       : static_cast<const __nv_bfloat16*>(a.w2) + (e * a.hidden + row0) * a.inter;
          const int64_t K = kUp ? a.hidden : a.inter;
          const int step = kBatch * fs.side;
          // once for every kFewRows pairs: the rows of more of them come again
          for (int pass = 0; pass < __popc(mine) && ok; pass += kFewRows)
            for (int i = 0; i < count; i += step) {
              if (rounds > 0 && !tc::mbar_wait(&sh->empty[at.stage], at.phase ^ 1u, kWaitLimit)) {
                ok = false;
                break;
              }
              const uint32_t bytes = (uint32_t)min(step, count - i) * fs.row_bytes;
              uint8_t* dst = smem + at.stage * fs.stage_bytes;
              tc::mbar_arrive_expect_tx(&sh->full[at.stage], kNR * bytes);
              bulk_load(dst, w + i * K, bytes, &sh->full[at.stage]);
              if (kUp) bulk_load(dst + step * fs.row_bytes, w + (i + (int64_t)a.inter) * K, bytes, &sh->full[at.stage]);
              at.next(fs.stages);
              rounds += at.stage == 0;
            }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      } else if (__popc(mine) == 1) {
        ok = few_expert<kUp, kP, 1>(a, fs, smem, sh, at, row0, count, mine, h, c0);
      } else {
        ok = few_expert<kUp, kP, kFewRows>(a, fs, smem, sh, at, row0, count, mine, h, c0);
      }
    }
    if (!ok && lane == 0) {
      atomicExch(&g_experts_error, producer ? 5 : 6);
      if (producer)  // copies in flight: those of this round, and of the one before it
        for (int s = 0; s < fs.stages; ++s)
          if (s < at.stage || rounds > 0) (void)tc::mbar_wait(&sh->full[s], s < at.stage ? at.phase : at.phase ^ 1u, kWaitLimit);
    }
  }
  if (kUp) return;
  __syncthreads();
  for (int i = threadIdx.x; i < (c1 - c0) * a.T; i += kFewThreads) {
    const int t = i / (c1 - c0), c = i - t * (c1 - c0);
    static_cast<__nv_bfloat16*>(a.out)[(int64_t)t * a.hidden + c0 + c] = __float2bfloat16_rn(sh->sum[c * kFewTokens + t]);
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* q = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &q, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(q);
    return nullptr;
  }();
  return fn;
}

// A bf16 tensor of `rank` dimensions, innermost first; strides in elements from the second on.
// Boxes of 64 channels in the 128-byte swizzle; what lies outside reads zero.
bool make_map(CUtensorMap* m, const void* base, int rank, const int64_t* dims, const int64_t* strides, const int* box) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t d[5], st[4];
  cuuint32_t b[5], es[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    b[i] = (cuuint32_t)box[i];
    es[i] = 1;
    if (i) st[i - 1] = (cuuint64_t)strides[i - 1] * 2;
  }
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), d, st, b, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kPass>
cudaError_t launch_gemm(const ExpertArgs& a, const void* rows, int64_t n, const int32_t* offs, void* out, cudaStream_t st) {
  GemmParams p{};
  p.N = kPass == 0 ? a.inter : a.hidden;
  p.K = kPass == 0 ? a.hidden : a.inter;
  p.E = a.E;
  p.rows = (int)n;
  p.limit = a.limit;
  p.offs = offs;
  p.out = out;
  CUtensorMap mw;
  RowMaps maps;
  bool ok;
  if (kPass == 0) {  // [E, 2, inter/16, 16, hidden] read as boxes of 16 gate rows, 16 up rows, four times
    const int64_t d[5] = {p.K, 16, 2, a.inter / 16, a.E};
    const int64_t s[4] = {p.K, (int64_t)a.inter * p.K, (int64_t)16 * p.K, (int64_t)2 * a.inter * p.K};
    const int b[5] = {kBK, 16, 2, 4, 1};
    ok = make_map(&mw, a.w13, 5, d, s, b);
  } else {
    const int64_t d[3] = {p.K, p.N, a.E}, s[2] = {p.K, (int64_t)p.N * p.K};
    const int b[3] = {kBK, 128, 1};
    ok = make_map(&mw, a.w2, 3, d, s, b);
  }
  const int64_t d[2] = {p.K, n}, s[1] = {p.K};
  for (int i = 0; i < kRowMaps; ++i) {
    const int b[2] = {kBK, 16 << i};
    ok = ok && make_map(&maps.box[i], rows, 2, d, s, b);
  }
  if (!ok) return cudaErrorInvalidValue;
  p.stages = gemm_smem(kStages, a.E) <= kSmemMost ? kStages : kStages - 1;  // 7 of up to 511 experts
  const size_t smem = gemm_smem(p.stages, a.E);
  // the same value in every call: another thread's may come between this and the launch
  cudaError_t e = cudaFuncSetAttribute(gemm_kernel<kPass>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMost);
  if (e != cudaSuccess) return e;
  return launch(gemm_kernel<kPass>, sm_count() / 2 * 2, kGemmThreads, smem, st, mw, maps, p);
}

}  // namespace

size_t expert_workspace_bytes(int64_t T, int hidden, int inter, int E, int topk) {
  return layout(T, hidden, inter, E, topk).total;
}

cudaError_t launch_experts(const ExpertArgs& a, cudaStream_t st) {
  const Layout l = layout(a.T, a.hidden, a.inter, a.E, a.topk);
  char* ws = static_cast<char*>(a.ws);
  int32_t* offs = reinterpret_cast<int32_t*>(ws + l.offs);
  int32_t* slot_row = reinterpret_cast<int32_t*>(ws + l.slot_row);
  __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(ws + l.h);
  float* yp = reinterpret_cast<float*>(ws + l.yp);
  __nv_bfloat16* xp = reinterpret_cast<__nv_bfloat16*>(yp);  // read before y is written
  const int64_t n = (int64_t)a.T * a.topk;
  cudaError_t e;
  if (n <= kFewPairs && a.T <= kFewTokens && a.hidden <= kFewWidth && a.inter <= kFewWidth) {
    const int grid = sm_count();
    const auto up = a.hidden <= kFewWidth / 2 ? few_kernel<true, 2> : few_kernel<true, 4>;
    const auto down = a.inter <= kFewWidth / 2 ? few_kernel<false, 2> : few_kernel<false, 4>;
    const size_t up_smem = kFewRing + sizeof(FewShared);
    const size_t down_smem = up_smem + (size_t)(a.hidden / grid + 1) * kFewTokens * 4;
    const size_t most = up_smem + (size_t)(kFewWidth / grid + 1) * kFewTokens * 4;  // of any call, see launch_gemm
    if ((e = cudaFuncSetAttribute(up, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(down, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most)) != cudaSuccess) return e;
    // both CTAs of an SM at once
    if ((e = cudaFuncSetAttribute(up, cudaFuncAttributePreferredSharedMemoryCarveout, 100)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(down, cudaFuncAttributePreferredSharedMemoryCarveout, 100)) != cudaSuccess) return e;
    float* h32 = reinterpret_cast<float*>(ws + l.h);
    if ((e = launch(up, grid, kFewThreads, up_smem, st, a, h32)) != cudaSuccess) return e;
    return launch(down, grid, kFewThreads, down_smem, st, a, h32);
  }
  const int pieces = (a.hidden / 8 + kPiece - 1) / kPiece, splits = a.T >= 2048 ? 1 : a.topk;
  const int64_t units = (int64_t)a.T * pieces * splits;
  if (n <= kPlaced) {
    e = launch(gather_kernel<true>, (units + a.E + kGatherWarps) / kGatherWarps, kGatherWarps * 32, 0, st, a, pieces, splits, offs, slot_row, xp);
  } else {
    if (n <= kOneCta) {
      e = launch(order_kernel, 1, kOrderThreads, 0, st, a.ids, n, n, a.E, nullptr, offs, slot_row);
    } else {
      const int64_t chunk = (n + kMaxChunks - 1) / kMaxChunks, chunks = (n + chunk - 1) / chunk;
      int32_t* counts = reinterpret_cast<int32_t*>(ws + l.counts);
      e = launch(count_kernel, chunks, kOrderThreads, 0, st, a.ids, n, chunk, a.E, counts);
      if (e != cudaSuccess) return e;
      e = launch(order_kernel, chunks, kOrderThreads, 0, st, a.ids, n, chunk, a.E, counts, offs, slot_row);
    }
    if (e != cudaSuccess) return e;
    e = launch(gather_kernel<false>, (units + kGatherWarps - 1) / kGatherWarps, kGatherWarps * 32, 0, st, a, pieces, splits, offs, slot_row, xp);
  }
  if (e != cudaSuccess) return e;
  if ((e = launch_gemm<0>(a, xp, n, offs, h, st)) != cudaSuccess) return e;
  if ((e = launch_gemm<1>(a, h, n, offs, yp, st)) != cudaSuccess) return e;
  // few tokens: a CTA per 1024 channels of one, many: a CTA per token (calls with small matrices, in us, with
  // parts and without: 8 x 4096 35.5 and 38.1, 64 x 8192 59.5 and 65.2, 1000 x 4096 93.3 and 91.7, 8192 x 4096
  // 520 and 505)
  const int parts = a.T >= 1024 ? 1 : (a.hidden / 4 + kCombineThreads - 1) / kCombineThreads;
  return launch(combine_kernel, (int64_t)a.T * parts, kCombineThreads, 0, st, a, parts, slot_row, yp);
}

cudaError_t take_experts_error(int* code) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_experts_error, sizeof(int));
  if (e != cudaSuccess) return e;
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_experts_error, &zero, sizeof(int));
  }
  *code = v;
  return e;
}

}  // namespace dsv4
