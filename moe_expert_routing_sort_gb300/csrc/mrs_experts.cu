// mrs_experts.cu -- the experts' products of MXFP4 rows and weights, driven by the sort step.
//
// For every row p of the sorted list that is a route r = sorted_token_ids[p] (r < T * topk), with
// e the owner of its block:
//   out[r, n] = w_p * sum over k of X[row(r), k] W[e, n, k],   row(r) = r, or r / topk
// X and W are E2M1 codes with one E8M0 scale per 32 columns; sums are fp32, the row's weight
// (1 without weights) is applied in fp32, and the result is rounded once to the output type.
#include <cuda_bf16.h>

#include "mrs_args.h"
#include "mrs_internal.h"
#include "mrs_mx.cuh"

namespace mrs {

struct ExpertsArgs {
  const unsigned char *xc, *xs, *wc, *ws;
  const int32_t* sid;
  const float* sw;  // or null
  const int32_t* eid;
  const int32_t* npp;
  int32_t* status;
  void* out;
  int routes, topk, per_route;
  int E, K, N, B, scols, max_rows;
};

constexpr int kExpThreads = 256;
constexpr int kExpRows = 16, kExpCols = 64, kExpK = 128;

// Simple form: 16 rows x 64 outputs per tile on the FMA pipes, operands decoded to fp32 in
// shared memory 128 columns at a time.
template <class Out>
__global__ void __launch_bounds__(kExpThreads) mrs_experts_kernel(const ExpertsArgs a) {
  __shared__ float xt[kExpRows][kExpK + 1];
  __shared__ float wt[kExpCols][kExpK + 1];
  __shared__ int rid[kExpRows];
  const int tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const int rows = min(max(__ldg(a.npp), 0), a.max_rows) / a.B * a.B;
  const int sub = min(a.B, kExpRows), subs = a.B / sub;
  const long long ntile = (a.N + kExpCols - 1) / kExpCols;
  const long long items = static_cast<long long>(rows / a.B) * subs * ntile;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int n0 = static_cast<int>(it % ntile) * kExpCols;
    const int p0 = static_cast<int>(it / ntile) * sub;
    const int e = __ldg(a.eid + p0 / a.B);
    if (e < 0 || e >= a.E) {
      if (tid == 0) atomicOr(a.status, MOE_RS_DEVICE_BAD_EXPERT_ID);
      continue;
    }
    __syncthreads();
    if (tid < kExpRows) {
      const int r = tid < sub ? __ldg(a.sid + p0 + tid) : -1;
      rid[tid] = (r >= 0 && r < a.routes) ? r : -1;
    }
    __syncthreads();
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < a.K; k0 += kExpK) {
      for (int q = tid; q < (kExpRows + kExpCols) * (kExpK / 8); q += kExpThreads) {
        const int r = q / (kExpK / 8), c = k0 + q % (kExpK / 8) * 8;
        float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        size_t row = 0;
        bool in = c < a.K;
        const bool isx = r < kExpRows;
        if (isx) {
          in = in && rid[r] >= 0;
          if (in) row = a.per_route ? rid[r] : rid[r] / a.topk;
        } else {
          in = in && n0 + r - kExpRows < a.N;
          row = static_cast<size_t>(e) * a.N + n0 + r - kExpRows;
        }
        if (in) {
          const unsigned char* codes = isx ? a.xc : a.wc;
          const unsigned char* scales = isx ? a.xs : a.ws;
          e2m1_values(__ldg(reinterpret_cast<const uint32_t*>(codes + row * (a.K / 2) + c / 2)), v);
          const float s = e8m0_value(__ldg(scales + row * a.scols + c / 32));
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= s;
        }
        float* dst = (isx ? &xt[r][0] : &wt[r - kExpRows][0]) + (c - k0);
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i] = v[i];
      }
      __syncthreads();
      for (int k = 0; k < kExpK; ++k) {
        const float x = xt[tid >> 4][k];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = fmaf(x, wt[(tid & 15) + 16 * j][k], acc[j]);
      }
      __syncthreads();
    }
    const int r = rid[tid >> 4];
    if (r >= 0) {
      const float w = a.sw ? __ldg(a.sw + p0 + (tid >> 4)) : 1.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + (tid & 15) + 16 * j;
        if (n >= a.N) continue;
        Out* o = static_cast<Out*>(a.out) + static_cast<size_t>(r) * a.N + n;
        if constexpr (sizeof(Out) == 4) *o = w * acc[j];
        else *o = __float2bfloat16_rn(w * acc[j]);
      }
    }
  }
}

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
  a.xc = x_codes;
  a.xs = x_scales;
  a.wc = w_codes;
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
  auto* k = out_dtype == MOE_RS_FP32 ? mrs_experts_kernel<float> : mrs_experts_kernel<__nv_bfloat16>;
  return launch_status(launch_pdl(k, dim3(4 * sms), dim3(kExpThreads), 0, stream, a));
}

}  // extern "C"
