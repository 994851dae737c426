// The experts' products of a routed layer:
//   out[t] = sum_j weights[t,j] * W2_e h,  h = silu(g) * u,  g = W1_e x_t,  u = W3_e x_t,  e = ids[t,j]
// with g <- min(g, limit) and u <- clamp(u, -limit, limit) when a limit is given.
// The (token, choice) pairs are put in order of their expert; h is rounded to bf16 (the type of
// the second product's operands), the products of a pair are kept in 32 bits until the sum over j.
#include <cuda.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "moe.h"
#include "tc_pair.cuh"

namespace dsv4 {

__device__ int g_experts_error = 0;

namespace {

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

// ---------------------------------------------------------------- the two products
//
// One kernel, a CTA pair per 256 x N tile: D[256 weight rows, N token rows] = W X^T, so that the
// ragged side (the rows of one expert) is N, which an MMA takes in steps of 16, and few rows cost
// little.  Each CTA of the pair holds 128 weight rows and half of the token rows.
//  * warp 0: TMA producer, kStages stages of 64 channels (16 KB of weights, up to 16 KB of rows).
//  * warp 1 (of the leader): M=256, K=16 MMAs into one of two 256-column accumulators, so that
//    a tile's epilogue overlaps the next tile's main loop.
//  * warps 2-5: epilogue, one TMEM lane quadrant each.
// First product (kPass 0): the TMA box interleaves 16 gate rows with 16 up rows, so that lanes l
// and l + 16 of an epilogue warp hold gate and up of one channel and one shuffle brings both
// together; h goes out in bf16.  Second product: y in fp32, a row of 32 channels per store.
// A tile's rows behind its expert's last one are the next expert's (or the fill's): their columns
// are computed and not stored.  Every wait is bounded; a role that gives up records
// g_experts_error and leaves, and the others time out behind it.
constexpr int kBK = 64, kStages = 6, kMaxN = 256;
constexpr uint32_t kStageA = 128 * kBK * 2, kStageB = (kMaxN / 2) * kBK * 2;
constexpr uint32_t kSmemData = kStages * (kStageA + kStageB);
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr int kGemmThreads = 192;

struct GemmParams {
  int N;        // output channels (inter, hidden)
  int K;        // reduction length
  int E;
  float limit;
  const int32_t* offs;  // [E+1] first row of each expert
  void* out;    // h (bf16) or y (fp32), [rows, N]
};

struct Bars {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
  uint32_t tmem_base;
};
constexpr uint32_t kSmemTotal = kSmemData + 1024;  // + barriers; the experts' offsets follow

// Walks the tiles of all experts in order: expert, then weight tile, then row tile.
struct Cursor {
  const int32_t* offs;
  int E, wt;                 // weight tiles of an expert
  int e = 0, n = 0, nt = 0;  // expert, its rows, its row tiles
  int64_t base = 0;          // tiles before expert e
  __device__ Cursor(const int32_t* o, int experts, int weight_tiles) : offs(o), E(experts), wt(weight_tiles) { open(); }
  __device__ void open() {
    n = e < E ? offs[e + 1] - offs[e] : 0;
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
    gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                const __grid_constant__ CUtensorMap map_x16, const __grid_constant__ GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = tc::cluster_cta_rank();
  Bars* bars = reinterpret_cast<Bars*>(smem + kSmemData);
  int32_t* offs = reinterpret_cast<int32_t*>(smem + kSmemTotal);
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
  for (int e = tid; e <= p.E; e += kGemmThreads) offs[e] = p.offs[e];
  if (warp == 1) {
    tc::tmem2_alloc(&bars->tmem_base, 512);
    tc::tmem2_relinquish();
  }
  if (tid == 0) {
    tc::prefetch_tensormap(&map_w);
    tc::prefetch_tensormap(&map_x);
    tc::prefetch_tensormap(&map_x16);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (!aligned) {
    if (tid == 0) atomicExch(&g_experts_error, 3);
  } else if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      Cursor cur(offs, p.E, weight_tiles);
      uint32_t it = 0;
      bool ok = true;
      int w, row, rows;
      for (int64_t t = pair; ok && cur.at(t, &w, &row, &rows); t += pairs) {
        const int half = (rows + 15) / 16 * 8;  // token rows of one CTA
        const int y = row + (int)rank * half;
        const int boxes = half > 64 ? 0 : (half + 15) / 16;  // one box of 128 rows, or boxes of 16
        const uint32_t bytes = kStageA + (boxes ? boxes * 16u : 128u) * kBK * 2;
        for (int k = 0; k < k_steps; ++k, ++it) {
          const int s = (int)(it % kStages);
          if (it >= kStages && !tc::mbar_wait(&bars->empty[s], ((it / kStages) - 1) & 1, kWaitLimit)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * (kStageA + kStageB);
          const uint32_t full = tc::cluster_addr(&bars->full[s], 0);
          if (rank == 0) tc::mbar_arrive_expect_tx(&bars->full[s], 2 * bytes);
          if (kPass == 0)
            tc::tma2_load_5d(sa, &map_w, k * kBK, 0, 0, w * 8 + (int)rank * 4, cur.e, full);
          else
            tc::tma2_load_3d(sa, &map_w, k * kBK, w * 256 + (int)rank * 128, cur.e, full);
          if (boxes == 0) tc::tma2_load_2d(sa + kStageA, &map_x, k * kBK, y, full);
          for (int b = 0; b < boxes; ++b)
            tc::tma2_load_2d(sa + kStageA + b * 16 * kBK * 2, &map_x16, k * kBK, y + 16 * b, full);
        }
      }
      if (!ok) {
        atomicExch(&g_experts_error, 1);
        for (uint32_t i = it < kStages ? 0 : it - kStages; rank == 0 && i < it; ++i)  // copies in flight
          (void)tc::mbar_wait(&bars->full[i % kStages], (i / kStages) & 1, kWaitLimit);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (the leader's)
    if (rank == 0 && lane == 0) {
      Cursor cur(offs, p.E, weight_tiles);
      uint32_t it = 0, lt = 0;
      bool ok = true;
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
        for (int k = 0; k < k_steps; ++k, ++it) {
          const int s = (int)(it % kStages);
          if (!tc::mbar_wait(&bars->full[s], (it / kStages) & 1, kWaitLimit)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint32_t a0 = tc::smem_u32(smem + s * (kStageA + kStageB));
          const uint64_t ad = tc::sdesc_sw128(a0, 16, 1024), bd = tc::sdesc_sw128(a0 + kStageA, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            tc::umma2_f16(acc, ad + 2 * kk, bd + 2 * kk, idesc, (k > 0 || kk > 0) ? 1u : 0u);
          tc::umma2_commit_both(&bars->empty[s]);  // free in both CTAs once these MMAs have read it
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

// Rows of x in order of their expert, as bf16.
__global__ void __launch_bounds__(256) gather_kernel(ExpertArgs a, const int32_t* offs, const int32_t* row_slot,
                                                     __nv_bfloat16* xp) {
  const int64_t r = blockIdx.x;
  if (r >= offs[a.E]) return;
  const int64_t t = row_slot[r] / a.topk;
  uint4* dst = reinterpret_cast<uint4*>(xp + r * a.hidden);
  const int n = a.hidden / 8;
  if (!a.x_scale) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + t * a.hidden);
    for (int i = threadIdx.x; i < n; i += 256) dst[i] = src[i];
    return;
  }
  const uint2* src = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + t * a.hidden);
  const float* sc = a.x_scale + t * ((a.hidden + kScaleGroup - 1) / kScaleGroup);
  for (int i = threadIdx.x; i < n; i += 256) {
    const uint2 q = src[i];
    const float s = sc[i / (kScaleGroup / 8)];
    uint4 o;
    uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)((j < 2 ? q.x : q.y) >> (16 * (j & 1)));
      const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
      const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    dst[i] = o;
  }
}

__global__ void __launch_bounds__(256) combine_kernel(ExpertArgs a, const int32_t* slot_row, const float* yp) {
  const int64_t t = blockIdx.x;
  for (int c = threadIdx.x; c < a.hidden; c += 256) {
    float s = 0.f;
    for (int j = 0; j < a.topk; ++j) {
      const int r = slot_row[t * a.topk + j];
      if (r >= 0) s += a.weights[t * a.topk + j] * yp[(int64_t)r * a.hidden + c];
    }
    static_cast<__nv_bfloat16*>(a.out)[t * a.hidden + c] = __float2bfloat16_rn(s);
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

int sm_count() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 148;
}

template <int kPass>
cudaError_t launch_gemm(const ExpertArgs& a, const void* rows, int64_t n, const int32_t* offs, void* out, cudaStream_t st) {
  GemmParams p{};
  p.N = kPass == 0 ? a.inter : a.hidden;
  p.K = kPass == 0 ? a.hidden : a.inter;
  p.E = a.E;
  p.limit = a.limit;
  p.offs = offs;
  p.out = out;
  CUtensorMap mw, mx, mx16;
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
  const int b[2] = {kBK, kMaxN / 2}, b16[2] = {kBK, 16};
  ok = ok && make_map(&mx, rows, 2, d, s, b) && make_map(&mx16, rows, 2, d, s, b16);
  if (!ok) return cudaErrorInvalidValue;
  const size_t smem = kSmemTotal + (size_t)(a.E + 1) * 4;
  cudaError_t e = cudaFuncSetAttribute(gemm_kernel<kPass>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  gemm_kernel<kPass><<<sm_count() / 2 * 2, kGemmThreads, smem, st>>>(mw, mx, mx16, p);
  note_launch(1);
  return cudaGetLastError();
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
  __nv_bfloat16* xp = reinterpret_cast<__nv_bfloat16*>(yp);  // read before y is written
  const int64_t n = (int64_t)a.T * a.topk;
  order_kernel<<<1, 1024, 0, st>>>(a.ids, n, a.E, offs, row_slot, slot_row);
  note_launch(1);
  gather_kernel<<<(unsigned)n, 256, 0, st>>>(a, offs, row_slot, xp);
  note_launch(1);
  cudaError_t e = launch_gemm<0>(a, xp, n, offs, h, st);
  if (e != cudaSuccess) return e;
  e = launch_gemm<1>(a, h, n, offs, yp, st);
  if (e != cudaSuccess) return e;
  combine_kernel<<<a.T, 256, 0, st>>>(a, slot_row, yp);
  note_launch(1);
  return cudaGetLastError();
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
