// mrs_experts.cu -- the experts' products of MXFP4 rows and weights, driven by the sort step.
//
// For every row p of the sorted list that is a route r = sorted_token_ids[p] (r < T * topk), with
// e the owner of its block:
//   out[r, n] = w_p * sum over k of X[row(r), k] W[e, n, k],   row(r) = r, or r / topk
// X and W are E2M1 codes with one E8M0 scale per 32 columns; sums are fp32, the row's weight
// (1 without weights) is applied in fp32, and the result is rounded once to the output type.
//
// One tile is 128 outputs of one expert (the M side of the tensor-core product: weights fill it
// whatever the number of tokens) by the rows of one block (the N side, BN = 16 .. 128; blocks of
// more rows are cut, blocks of fewer leave columns unused).  A persistent CTA per SM takes tiles
// round robin, the output tiles of a block next to each other, so the SMs share a block's rows
// and an expert's weights in L2.  Steps of 256 columns (128 bytes a row) go through a ring of
// shared-memory stages; the warps of a CTA each have one task:
//   0     tensor copies: the weights' tile, and the block's rows gathered by index four at a
//         time, both in the 128-byte swizzle the tensor core reads
//   1     one thread copies the step's scales to tensor memory and issues four products of 64
//         columns; the tensor core applies the scales and adds into fp32 in tensor memory
//   2, 3  scales of the weights and of the rows, from row-major bytes to the order that tensor
//         memory wants (row r of 128: lane r % 32, word r / 32 of 4 scales)
//   4-7   a finished tile from tensor memory to the output rows, while the next one is computed
//         (two accumulators)
// Every wait is bounded; a wait that gives up ends its warp's task with the status bit set, and
// the CTA leaves once nothing of its own is in flight.
#include <type_traits>

#include <cuda_bf16.h>

#include "mrs_args.h"
#include "mrs_internal.h"
#include "mrs_tc.cuh"

namespace mrs {

struct ExpertsArgs {
  const unsigned char *xs, *ws;  // scales
  const int32_t* sid;
  const float* sw;  // or null
  const int32_t* eid;
  const int32_t* npp;
  int32_t* status;
  void* out;
  unsigned long long wait_limit_ns;
  int routes, topk, per_route;
  int E, K, N, B, scols, max_rows;
  int sub, subs;   // rows of a tile (<= BN), tiles along a block's rows
  int ntile;       // tiles along the outputs
  int ksteps;      // steps of 256 columns
};

constexpr int kExpThreads = 256;
constexpr int kExpM = 128;           // outputs per tile
constexpr int kStepBytes = 128;      // bytes of a row per step
constexpr int kScaleBytes = 2048;    // weights' and rows' scales of a step: 2 x 2 x 512
constexpr int kTmemCols = 512;
constexpr int kScalePrefetch = 4;    // steps whose scales a warp keeps in flight

template <int BN>
struct ExpertsStage {
  static constexpr int kA = kExpM * kStepBytes;
  static constexpr int kB = BN * kStepBytes;
  static constexpr int kBytes = kA + kB + kScaleBytes;
  // as many as fit beside the barriers, at most 10
  static constexpr int kFit = (227 * 1024 - 2048) / kBytes;
  static constexpr int kStages = kFit < 10 ? kFit : 10;
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kBytes + 1024;
};

struct ExpertsTile {
  int p0, n0, e;
};

// Tile `it` of the list; false if its block's expert id is none (every warp decides alike).
__device__ __forceinline__ bool experts_tile(const ExpertsArgs& a, long long it, ExpertsTile& t) {
  const int b = static_cast<int>(it / a.ntile);
  t.n0 = static_cast<int>(it - static_cast<long long>(b) * a.ntile) * kExpM;
  t.p0 = b * a.sub;
  t.e = __ldg(a.eid + b / a.subs);
  return t.e >= 0 && t.e < a.E;
}

// Row i of the tile: its route, or -1 (padding, an entry outside the routes, a column unused).
__device__ __forceinline__ int experts_route(const ExpertsArgs& a, const ExpertsTile& t, int i) {
  if (i >= a.sub) return -1;
  const int r = __ldg(a.sid + t.p0 + i);
  return r >= 0 && r < a.routes ? r : -1;
}

// Scales of a warp's rows (lane + 32 j of the tile) for step `ks`: word j of q[g] holds the four
// bytes of row lane + 32 j at columns [256 ks + 128 g, + 128).  Null rows and bytes past the
// `blocks` scales of a row give 0, a finite scale, whatever the padding holds.
__device__ __forceinline__ void load_scales(const unsigned char* const (&row)[4], int ks,
                                            int blocks, uint4 (&q)[2]) {
  uint32_t w[2][4];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int at = 8 * ks + 4 * g, left = blocks - at;
    const uint32_t keep = left >= 4 ? ~0u : (1u << (8 * max(left, 0))) - 1u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[g][j] = (row[j] != nullptr && left > 0)
                    ? __ldg(reinterpret_cast<const uint32_t*>(row[j] + at)) & keep
                    : 0u;
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) q[g] = make_uint4(w[g][0], w[g][1], w[g][2], w[g][3]);
}

template <int BN, class Out>
__global__ void __launch_bounds__(kExpThreads, 1)
    mrs_experts_kernel(const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap xmap, const ExpertsArgs a) {
  using St = ExpertsStage<BN>;
  constexpr int S = St::kStages;
  extern __shared__ unsigned char smem_raw[];
  __shared__ unsigned long long full_s[S], scaled_s[S], empty_s[S], acc_full_s[2], acc_free_s[2],
      done_s;
  __shared__ uint32_t tmem_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const unsigned long long limit = a.wait_limit_ns;
  pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full_s[s], 1);
      mbar_init(&scaled_s[s], 2);
      mbar_init(&empty_s[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full_s[b], 1);
      mbar_init(&acc_free_s[b], 4);
    }
    mbar_init(&done_s, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_s, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  pdl_wait();

  const int rows = min(max(__ldg(a.npp), 0), a.max_rows);
  const long long tiles = static_cast<long long>(rows / a.B) * a.subs * a.ntile;
  ExpertsTile t;
  bool ok = true;
  int stage = 0;
  uint32_t phase = 0;  // parity of the ring's current round
  auto advance = [&] {
    if (++stage == S) {
      stage = 0;
      phase ^= 1u;
    }
  };

  if (warp == 0) {
    long long issued = 0;
    for (long long it = blockIdx.x; ok && it < tiles; it += gridDim.x) {
      if (!experts_tile(a, it, t)) {
        if (lane == 0) atomicOr(a.status, MOE_RS_DEVICE_BAD_EXPERT_ID);
        continue;
      }
      int row[4] = {0, 0, 0, 0};  // rows that are no route read row 0, and are not stored
      if (4 * lane < BN) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = experts_route(a, t, 4 * lane + j);
          row[j] = r < 0 ? 0 : (a.per_route ? r : r / a.topk);
        }
      }
      for (int ks = 0; ks < a.ksteps; ++ks) {
        ok = mbar_wait_bounded(&empty_s[stage], phase ^ 1u, limit);
        if (!ok) break;
        const uint32_t dst = base + stage * St::kBytes;
        if (lane == 0) {
          mbar_expect(&full_s[stage], St::kA + St::kB);
          tma_load_3d(dst, &wmap, ks * kStepBytes, t.n0, t.e, &full_s[stage]);
        }
        __syncwarp();
        if (4 * lane < BN)
          tma_gather4(dst + St::kA + lane * 4 * kStepBytes, &xmap, ks * kStepBytes, row[0], row[1],
                      row[2], row[3], &full_s[stage]);
        __syncwarp();
        ++issued;
        advance();
      }
    }
    if (!ok) {
      // copies still on their way must land before the CTA leaves: the last S issued
      for (long long q = issued > S ? issued - S : 0; q < issued; ++q)
        mbar_wait_bounded(&full_s[q % S], static_cast<uint32_t>(q / S) & 1u, kWaitLimitNs);
    }
  } else if (warp == 1) {
    int buf = 0;
    uint32_t acc_phase = 0;
    bool any = false;
    for (long long it = blockIdx.x; ok && it < tiles; it += gridDim.x) {
      if (!experts_tile(a, it, t)) continue;
      ok = mbar_wait_bounded(&acc_free_s[buf], acc_phase ^ 1u, limit);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + buf * BN;
      for (int ks = 0; ks < a.ksteps; ++ks) {
        ok = mbar_wait_bounded(&full_s[stage], phase, limit) &&
             mbar_wait_bounded(&scaled_s[stage], phase, limit);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t src = base + stage * St::kBytes, sc = src + St::kA + St::kB;
          const uint32_t ts = tmem + 2 * BN + stage * 16;
          const uint64_t da = desc_rows128(src), db = desc_rows128(src + St::kA);
          const int parts = min(4, (a.K - 256 * ks + 63) >> 6);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            tc_copy_scales(ts + 4 * g, desc_scales(sc + 512 * g));
            tc_copy_scales(ts + 8 + 4 * g, desc_scales(sc + 1024 + 512 * g));
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q >= parts) break;  // columns past K
            // 32 bytes further along the swizzled rows: 2 units of 16
            tc_mma_mxf4(d, da + 2 * q, db + 2 * q, mxf4_word(kExpM, BN, (q & 1) * 2),
                        ts + 4 * (q >> 1), ts + 8 + 4 * (q >> 1), ks > 0 || q > 0);
          }
          tc_commit(&empty_s[stage]);
          if (ks + 1 == a.ksteps) tc_commit(&acc_full_s[buf]);
        }
        any = true;
        __syncwarp();
        advance();
      }
      buf ^= 1;
      if (buf == 0) acc_phase ^= 1u;
    }
    // nothing of the tensor core may be in flight when tensor memory is given back
    if (any) {
      if (lane == 0) tc_commit(&done_s);
      __syncwarp();
      mbar_wait_bounded(&done_s, 0, kWaitLimitNs);
    }
  } else if (warp < 4) {
    const bool weights = warp == 2;
    for (long long it = blockIdx.x; ok && it < tiles; it += gridDim.x) {
      if (!experts_tile(a, it, t)) continue;
      const unsigned char* row[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = lane + 32 * j;
        row[j] = nullptr;
        if (weights) {
          if (t.n0 + i < a.N)
            row[j] = a.ws + (static_cast<size_t>(t.e) * a.N + t.n0 + i) * a.scols;
        } else if (i < BN) {
          const int r = experts_route(a, t, i);
          if (r >= 0) row[j] = a.xs + static_cast<size_t>(a.per_route ? r : r / a.topk) * a.scols;
        }
      }
      uint4 q[kScalePrefetch][2], n[kScalePrefetch][2];
#pragma unroll
      for (int c = 0; c < kScalePrefetch; ++c) load_scales(row, c, a.K / 32, n[c]);
      for (int k0 = 0; ok && k0 < a.ksteps; k0 += kScalePrefetch) {
#pragma unroll
        for (int c = 0; c < kScalePrefetch; ++c) {
          q[c][0] = n[c][0];
          q[c][1] = n[c][1];
          load_scales(row, k0 + kScalePrefetch + c, a.K / 32, n[c]);
        }
#pragma unroll
        for (int c = 0; c < kScalePrefetch; ++c) {
          if (k0 + c >= a.ksteps) break;
          ok = mbar_wait_bounded(&empty_s[stage], phase ^ 1u, limit);
          if (!ok) break;
          const uint32_t dst = base + stage * St::kBytes + St::kA + St::kB + (weights ? 0 : 1024) +
                               16 * lane;
#pragma unroll
          for (int g = 0; g < 2; ++g)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 512 * g),
                         "r"(q[c][g].x), "r"(q[c][g].y), "r"(q[c][g].z), "r"(q[c][g].w)
                         : "memory");
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&scaled_s[stage]);
          advance();
        }
      }
    }
  } else {
    const int quarter = warp - 4;
    int buf = 0;
    uint32_t acc_phase = 0;
    for (long long it = blockIdx.x; ok && it < tiles; it += gridDim.x) {
      if (!experts_tile(a, it, t)) continue;
      constexpr int NJ = (BN + 31) / 32;
      int route[NJ];
      float weight[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int i = lane + 32 * j;
        route[j] = experts_route(a, t, i);
        weight[j] = (a.sw != nullptr && route[j] >= 0) ? __ldg(a.sw + t.p0 + i) : 1.0f;
      }
      ok = mbar_wait_bounded(&acc_full_s[buf], acc_phase, limit);
      if (!ok) break;
      tc_fence_after();
      const int n = t.n0 + 32 * quarter + lane;
      const uint32_t src = tmem + buf * BN + (static_cast<uint32_t>(32 * quarter) << 16);
#pragma unroll
      for (int c0 = 0; c0 < BN; c0 += 16) {
        float v[16];
        tmem_load16(src + c0, v);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const int r = __shfl_sync(kFull, route[(c0 + c) >> 5], (c0 + c) & 31);
          const float w = __shfl_sync(kFull, weight[(c0 + c) >> 5], (c0 + c) & 31);
          if (r < 0 || n >= a.N) continue;
          Out* o = static_cast<Out*>(a.out) + static_cast<size_t>(r) * a.N + n;
          if constexpr (sizeof(Out) == 4) *o = w * v[c];
          else *o = __float2bfloat16_rn(w * v[c]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_free_s[buf]);
      buf ^= 1;
      if (buf == 0) acc_phase ^= 1u;
    }
  }
  if (!ok && lane == 0) atomicOr(a.status, MOE_RS_DEVICE_WAIT_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free(tmem, kTmemCols);
}

// ------------------------------------------------------------------------------ host side
namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Bytes in rows of `row` bytes, `n1` rows a matrix, `n2` matrices; the copied box is 128 bytes of
// `box1` rows of one matrix.
bool encode_rows(CUtensorMap* map, const void* p, size_t row, size_t n1, size_t n2, int box1,
                 int rank) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {row, n1, n2};
  const cuuint64_t strides[2] = {row, row * n1};
  const cuuint32_t box[3] = {kStepBytes, static_cast<cuuint32_t>(box1), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(rank),
            const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, class Out>
cudaError_t launch_experts(const CUtensorMap& wmap, const CUtensorMap& xmap, const ExpertsArgs& a,
                           int grid, cudaStream_t st) {
  auto* k = mrs_experts_kernel<BN, Out>;
  const size_t smem = ExpertsStage<BN>::kSmem;
  const cudaError_t err =
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  return launch_pdl(k, dim3(grid), dim3(kExpThreads), smem, st, wmap, xmap, a);
}

}  // namespace

}  // namespace mrs

using namespace mrs;

extern "C" {

size_t moe_experts_mxfp4_workspace_bytes(int T, int E, int topk, int block_m) {
  if (T < 0 || E < 1 || E > kMaxExperts || topk < 1 || topk > kMaxTopk || block_m < 1 ||
      block_m > 1024 || (block_m & (block_m - 1)) != 0)
    return 0;
  return 256;
}

int moe_experts_mxfp4(const uint8_t* x_codes, const uint8_t* x_scales, int x_per_route,
                      const uint8_t* w_codes, const uint8_t* w_scales, int T, int E, int topk,
                      int cols, int outs, int block_m, const int32_t* sorted_token_ids,
                      const float* sorted_weights, const int32_t* expert_ids,
                      const int32_t* num_tokens_post_pad, void* out, int out_dtype,
                      void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (T < 0) return MOE_RS_ERR_BAD_TOKENS;
  if (E < 1 || E > kMaxExperts) return MOE_RS_ERR_BAD_EXPERTS;
  if (topk < 1 || topk > kMaxTopk) return MOE_RS_ERR_BAD_TOPK;
  const size_t need = moe_experts_mxfp4_workspace_bytes(T, E, topk, block_m);
  if (need == 0) return MOE_RS_ERR_BAD_BLOCK_M;
  const int scols = moe_mxfp4_scale_cols(cols);
  if (scols == 0 || outs < 8 || outs > MOE_RS_MXFP4_MAX_OUTS || outs % 8 != 0)
    return MOE_RS_ERR_BAD_COLS;
  if (out_dtype != MOE_RS_BF16 && out_dtype != MOE_RS_FP32) return MOE_RS_ERR_BAD_DTYPE;
  if (static_cast<int64_t>(T) * topk > INT32_MAX ||
      static_cast<int64_t>(moe_sort_max_padded(T, E, topk, block_m)) > INT32_MAX)
    return MOE_RS_ERR_OVERFLOW;
  if (!workspace || workspace_bytes < need) return MOE_RS_ERR_WORKSPACE;
  if (T == 0) return MOE_RS_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !sorted_token_ids || !expert_ids ||
      !num_tokens_post_pad || !out)
    return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(x_codes, 16) || !aligned(w_codes, 16) || !aligned(x_scales, 4) ||
      !aligned(w_scales, 4) || !aligned(sorted_token_ids, 4) || !aligned(sorted_weights, 4) ||
      !aligned(expert_ids, 4) || !aligned(num_tokens_post_pad, 4) || !aligned(out, 16) ||
      !aligned(workspace, 16))
    return MOE_RS_ERR_MISALIGNED;
  const size_t routes = static_cast<size_t>(T) * topk;
  const size_t xrows = x_per_route ? routes : static_cast<size_t>(T);
  const size_t wrows = static_cast<size_t>(E) * outs;
  const size_t P = moe_sort_max_padded(T, E, topk, block_m);
  const Span outs_s[] = {span(out, routes * outs * (out_dtype == MOE_RS_FP32 ? 4 : 2)),
                         span(workspace, workspace_bytes)};
  const Span ins[] = {span(x_codes, xrows * (cols / 2)),
                      span(x_scales, xrows * scols),
                      span(w_codes, wrows * (cols / 2)),
                      span(w_scales, wrows * scols),
                      span(sorted_token_ids, 4 * P),
                      span(sorted_weights, sorted_weights ? 4 * P : 0),
                      span(expert_ids, 4 * (P / block_m)),
                      span(num_tokens_post_pad, 4)};
  if (any_alias(outs_s, 2, ins, 8)) return MOE_RS_ERR_ALIAS;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return launch_status(cudaErrorInvalidDevice);
  ExpertsArgs a{};
  a.xs = x_scales;
  a.ws = w_scales;
  a.sid = sorted_token_ids;
  a.sw = sorted_weights;
  a.eid = expert_ids;
  a.npp = num_tokens_post_pad;
  a.status = static_cast<int32_t*>(workspace);
  a.out = out;
  a.routes = static_cast<int>(routes);
  a.topk = topk;
  a.per_route = x_per_route != 0;
  a.E = E;
  a.K = cols;
  a.N = outs;
  a.B = block_m;
  a.scols = scols;
  a.max_rows = static_cast<int>(P);
  a.wait_limit_ns = debug_wait_limit_ns();
  const int bn = block_m <= 16 ? 16 : (block_m >= 128 ? 128 : block_m);
  a.sub = block_m < bn ? block_m : bn;
  a.subs = block_m / a.sub;
  a.ntile = (outs + kExpM - 1) / kExpM;
  a.ksteps = (cols + 255) / 256;
  CUtensorMap wmap, xmap;
  if (!encode_rows(&wmap, w_codes, cols / 2, outs, E, kExpM, 3) ||
      !encode_rows(&xmap, x_codes, cols / 2, xrows, 1, 1, 2))
    return MOE_RS_ERR_LAUNCH;
  const int64_t tiles = static_cast<int64_t>(P / block_m) * a.subs * a.ntile;
  const int grid = tiles < sms ? static_cast<int>(tiles) : sms;
  const bool f32 = out_dtype == MOE_RS_FP32;
  auto go = [&](auto n) {
    constexpr int BN = decltype(n)::value;
    return f32 ? launch_experts<BN, float>(wmap, xmap, a, grid, stream)
               : launch_experts<BN, __nv_bfloat16>(wmap, xmap, a, grid, stream);
  };
  using std::integral_constant;
  return launch_status(bn == 16   ? go(integral_constant<int, 16>{})
                       : bn == 32 ? go(integral_constant<int, 32>{})
                       : bn == 64 ? go(integral_constant<int, 64>{})
                                  : go(integral_constant<int, 128>{}));
}

}  // extern "C"
