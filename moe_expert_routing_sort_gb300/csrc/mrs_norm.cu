// mrs_norm.cu -- root-mean-square norm of the residual plus a token's expert rows, and its gradient.
//
// Per token t, over c < cols, with x rows t * parts + j of the experts' products:
//   s[c]  = round16(residual[c] + x_0[c] + ... + x_{parts-1}[c])      sums in fp32, in this order
//   rstd  = 1 / sqrt(mean of s^2 + eps)
//   y[c]  = s[c] * gain[c] * rstd         to 16 bits, and / or to e4m3 with the row's scale
// The norm is that of the rounded s, which is what the next layer and the gradient read.  The
// 8-bit row is made from the fp32 y, not from its 16-bit rounding.  |y| is largest where |s * gain|
// is, so the scale and rstd come from one reduction.
//
// Gradient, d = grad + grad_rows_0 + ... + grad_rows_{parts-1}, xh = s * rstd, g = d * gain:
//   grad_x[c]    = rstd * (g - xh * mean of g * xh) + grad_sum[c]
//   grad_gain[c] = sum over tokens of d * xh
// grad_x is the gradient of the residual and of each of the token's rows.  A CTA keeps its columns'
// sums in registers over its tokens (a block of 32 tokens at a time, so that sums stay short) and
// leaves one row of partial sums; a second kernel adds these in a fixed order.
//
// Bound by memory: one read of every row, one write of every result.  The rows come through shared
// memory ahead of their use (RowStream), two vectors a thread, and the gain stays in registers.
// 8192 rows of 3584 in fp16, residual and one part, 16-bit and 8-bit results: 48.8 us, 80 % of the
// rate of a copy; what is left is issue (58 % of the slots) and the two meetings of a row's warps.
// Gradient, 8192 rows of 7168, 8 parts: 229 us, 90 %.  One token of 16 rows of 3584: 4.6 to 5.0 us in a
// graph, most of it the launch and one round trip to memory.
// Not in registers alone: two vectors a thread with a bound of 1024 threads leave 64 registers.  The
// gradient keeps 392 bytes of a thread in local memory for rows of 392 to 512 columns, 80 up to 7168, 208
// above; the norm 96 where a CTA has several rows.  Gradient of 8192 rows, 8 parts, each call by itself:
// 512 columns 80 us of 15, 3584 133 of 104, 7168 238 of 207, 8192 281 of 237; the norm with a residual 14
// of 5, 45 of 35, 84 of 69, 96 of 79.
#include "mrs_rows.cuh"

namespace mrs {

struct NormArgs {
  const void *x, *residual, *gain;
  size_t x_stride, residual_stride;
  int64_t rows;
  int parts, vecs, tpr, per_cta, gain_f32;
  float eps, inv_cols;
  void *y, *sum;
  unsigned char* codes;
  float *scales, *rstd;
};

// kOne: a row takes the whole CTA.
template <class T, int kVec, int kDepth, bool kOne>
__global__ void __launch_bounds__(kRowThreads<kVec>) mrs_norm_kernel(const NormArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ RowTotals meet[32];
  pdl_trigger();
  const int tid = threadIdx.x, in_cta = kOne ? 0 : tid / a.tpr, place = tid - in_cta * a.tpr;
  const int per_cta = kOne ? 1 : a.per_cta;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * per_cta + in_cta;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per_cta;
  const size_t row_bytes = 16 * static_cast<size_t>(a.vecs);
  RowStream<kVec, kDepth> stream(smem_raw, place, a.tpr, a.vecs);
  pdl_wait();
  // a token's items: its rows behind the residual, if there is one
  const bool lead = a.residual != nullptr;
  const unsigned char* next_x = static_cast<const unsigned char*>(a.x) +
                                2 * static_cast<size_t>(first) * a.parts * a.x_stride;
  const unsigned char* next_r =
      static_cast<const unsigned char*>(a.residual) + 2 * first * a.residual_stride;
  int64_t ahead = first;
  int item = lead ? -1 : 0;
  auto put = [&] {
    stream.put(ahead < a.rows, item < 0 ? next_r : next_x);
    if (item >= 0) next_x += 2 * a.x_stride;
    if (++item == a.parts) {
      item = lead ? -1 : 0;
      ahead += step;
      next_x += 2 * static_cast<size_t>(step - 1) * a.parts * a.x_stride;
      next_r += 2 * step * a.residual_stride;
    }
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) put();
  F2 gain[kVec][4];  // every row's
#pragma unroll
  for (int i = 0; i < kVec; ++i)
    if (i < stream.count) load_columns<T>(a.gain, a.gain_f32 != 0, i * a.tpr + place, gain[i]);
  // (the rows of a CTA take the same number of turns: they meet in the reduction)
  for (int64_t row = first; row - in_cta < a.rows; row += step) {
    const bool live = row < a.rows;
    F2 v[kVec][4];
    uint4 q[kVec];
    put();
    stream.get(q);
#pragma unroll
    for (int i = 0; i < kVec; ++i) unpack8<T>(q[i], v[i]);
    for (int j = lead ? 0 : 1; j < a.parts; ++j) {
      put();
      stream.get(q);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        F2 p[4];
        unpack8<T>(q[i], p);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i][k] = v[i][k] + p[k];
      }
    }
    F2 squares = f2(0.0f, 0.0f);
    float top = 0.0f;
    const size_t here = row * row_bytes;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (!live || i >= stream.count) continue;  // (what was read there is not of this row)
      const uint4 s = pack8<T>(v[i]);
      unpack8<T>(s, v[i]);
      if (a.sum != nullptr)
        *reinterpret_cast<uint4*>(static_cast<unsigned char*>(a.sum) + here + stream.off[i]) = s;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        squares = f2_fma(v[i][k], v[i][k], squares);
        v[i][k] = v[i][k] * gain[i][k];
      }
      if (a.codes != nullptr) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 p = f2_pair(v[i][k]);
          top = larger(larger(top, p.x), p.y);
        }
      }
    }
    const RowTotals r = row_totals(f2_sum(squares), __float_as_uint(top), a.tpr, meet);
    const float rstd = __frsqrt_rn(r.sum * a.inv_cols + a.eps);
    const float scale = fp8_scale(magnitude(__uint_as_float(r.top) * rstd));
    if (live && place == 0) {
      if (a.rstd != nullptr) a.rstd[row] = rstd;
      if (a.scales != nullptr) a.scales[row] = scale;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (!live || i >= stream.count) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][k] = v[i][k] * f2(rstd, rstd);
      if (a.y != nullptr)
        *reinterpret_cast<uint4*>(static_cast<unsigned char*>(a.y) + here + stream.off[i]) =
            pack8<T>(v[i]);
      if (a.codes != nullptr)
        *reinterpret_cast<uint2*>(a.codes + (here + stream.off[i]) / 2) = fp8_codes_of(v[i], scale);
    }
  }
}

struct NormGradArgs {
  const void *s, *gain, *grad, *grad_rows, *grad_sum;
  const float* rstd;
  int64_t rows;
  int parts, vecs, tpr, per_cta, gain_f32;
  float inv_cols;
  void* grad_x;
  float* partial;  // [CTAs * per_cta, cols], or null
};

constexpr int kNormSumRows = 32;

// kThreads: of the CTA at most, and two such CTAs an SM where that is below 512.
template <class T, int kVec, bool kOne, int kThreads = kRowThreads<kVec>>
__global__ void __launch_bounds__(kThreads, kThreads < 512 && kOne ? 2 : 1)
    mrs_norm_grad_kernel(const NormGradArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ RowTotals meet[32];
  pdl_trigger();
  const int tid = threadIdx.x, in_cta = kOne ? 0 : tid / a.tpr, place = tid - in_cta * a.tpr;
  const int per_cta = kOne ? 1 : a.per_cta;
  const size_t row_bytes = 16 * static_cast<size_t>(a.vecs), cols = 8 * static_cast<size_t>(a.vecs);
  const int64_t step = static_cast<int64_t>(gridDim.x) * per_cta;
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * per_cta;
  RowStream<kVec, kRowDepth<kVec>> stream(smem_raw, place, a.tpr, a.vecs);
  pdl_wait();
  // a token's items: s, grad, its rows, grad_sum, those that there are
  const int rows_of = a.grad_rows != nullptr ? a.parts : 0, behind = a.grad != nullptr ? 2 : 1;
  const int summed = behind + rows_of, items = summed + (a.grad_sum != nullptr ? 1 : 0);
  int64_t ahead = begin + in_cta;
  size_t token = ahead * row_bytes;
  const unsigned char* next_rows = static_cast<const unsigned char*>(a.grad_rows) + token * a.parts;
  int item = 0;
  auto put = [&] {
    const bool of_rows = item >= behind && item < summed;
    const void* base = item == 0 ? a.s : (item < behind ? a.grad : a.grad_sum);
    stream.put(ahead < a.rows,
               of_rows ? next_rows : static_cast<const unsigned char*>(base) + token);
    if (of_rows) next_rows += row_bytes;
    if (++item == items) {
      item = 0;
      ahead += step;
      token += step * row_bytes;
      next_rows += static_cast<size_t>(step - 1) * a.parts * row_bytes;
    }
  };
#pragma unroll
  for (int i = 0; i < kRowDepth<kVec> - 1; ++i) put();
  // Column sums: 32 tokens' at a time in registers, those behind the items in shared memory.
  F2 near[kVec][4];
  float4* far = reinterpret_cast<float4*>(
                    smem_raw + RowStream<kVec, kRowDepth<kVec>>::bytes(blockDim.x)) + tid;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
#pragma unroll
    for (int k = 0; k < 4; ++k) near[i][k] = f2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < 2; ++k) far[(2 * i + k) * blockDim.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  auto add_far = [&] {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float4& f = far[(2 * i + k) * blockDim.x];
        const float2 lo = f2_pair(near[i][2 * k]), hi = f2_pair(near[i][2 * k + 1]);
        f = make_float4(f.x + lo.x, f.y + lo.y, f.z + hi.x, f.w + hi.y);
        near[i][2 * k] = near[i][2 * k + 1] = f2(0.0f, 0.0f);
      }
  };
  int added = 0;
  // (a CTA's rows take the same number of turns: they meet in the reduction)
  for (int64_t first = begin; first < a.rows; first += step) {
    const int64_t row = first + in_cta;
    const bool live = row < a.rows;
    const float rstd = live ? __ldg(a.rstd + row) : 0.0f;
    F2 g[kVec][4], dot2 = f2(0.0f, 0.0f);
    uint4 s[kVec], q[kVec];
    put();
    stream.get(s);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) g[i][k] = f2(0.0f, 0.0f);
    for (int j = 1; j < summed; ++j) {
      put();
      stream.get(q);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        F2 p[4];
        unpack8<T>(q[i], p);
#pragma unroll
        for (int k = 0; k < 4; ++k) g[i][k] = g[i][k] + p[k];
      }
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (!live || i >= stream.count) continue;  // (what was read there is not of this row)
      F2 w[4], xh[4];
      load_columns<T>(a.gain, a.gain_f32 != 0, i * a.tpr + place, w);
      unpack8<T>(s[i], xh);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        xh[k] = xh[k] * f2(rstd, rstd);
        near[i][k] = f2_fma(g[i][k], xh[k], near[i][k]);
        g[i][k] = g[i][k] * w[k];
        dot2 = f2_fma(g[i][k], xh[k], dot2);
      }
    }
    const float mean = row_totals(f2_sum(dot2), 0u, a.tpr, meet).sum * a.inv_cols;
    if (a.grad_sum != nullptr) {
      put();
      stream.get(q);
    }
    const F2 by = f2(rstd, rstd), less = f2(-mean * rstd, -mean * rstd);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (!live || i >= stream.count) continue;
      F2 d[4], x[4];
      unpack8<T>(s[i], x);
      if (a.grad_sum != nullptr) unpack8<T>(q[i], d);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const F2 u = f2_fma(x[k], less, g[i][k]);  // g - xh * mean
        d[k] = a.grad_sum != nullptr ? f2_fma(u, by, d[k]) : u * by;
      }
      *reinterpret_cast<uint4*>(static_cast<unsigned char*>(a.grad_x) + row * row_bytes +
                                stream.off[i]) = pack8<T>(d);
    }
    if (++added == kNormSumRows) {
      added = 0;
      add_far();
    }
  }
  if (a.partial == nullptr) return;
  add_far();
  float* out = a.partial + (static_cast<size_t>(blockIdx.x) * a.per_cta + in_cta) * cols;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    if (i >= stream.count) continue;
    float4* p = reinterpret_cast<float4*>(out + stream.off[i] / 2);
    p[0] = far[2 * i * blockDim.x];
    p[1] = far[(2 * i + 1) * blockDim.x];
  }
}

// Column sums of `n` rows: a CTA has 32 columns, its 8 warps every eighth row each.
__global__ void __launch_bounds__(256) mrs_norm_gain_kernel(const float* partial, int n, int cols,
                                                            float* out) {
  __shared__ float meet[8][32];
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = 32 * blockIdx.x + lane;
  pdl_wait();
  float sum = 0.0f;
  if (c < cols) {
#pragma unroll 4
    for (int r = warp; r < n; r += 8) sum += partial[static_cast<size_t>(r) * cols + c];
  }
  meet[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && c < cols) {
#pragma unroll
    for (int w = 1; w < 8; ++w) sum += meet[w][lane];
    out[c] = sum;
  }
}

namespace {

// CTAs of the gradient on a device of `sms` SMs, for a workspace that does not know the device.
constexpr int kNormMaxSms = 256;
int norm_grad_ctas(const RowPlan& p, int sms) {
  const int per_sm = 1024 / p.threads;
  return sms * (per_sm < 1 ? 1 : per_sm);
}
RowPlan norm_grad_plan(int cols) { return row_plan(cols, 2, 128); }

constexpr int kNormDeepThreads = 640;  // of CTAs with twice as many items ahead
constexpr int kNormTwoThreads = 448;   // of the gradient's CTAs that share an SM, 72 registers each

template <class T, int kVec, int kDepth, bool kOne>
cudaError_t launch_norm(const NormArgs& a, const RowPlan& p, int sms, cudaStream_t st) {
  auto* k = mrs_norm_kernel<T, kVec, kDepth, kOne>;
  const size_t smem = RowStream<kVec, kDepth>::bytes(p.threads);
  constexpr int most_threads = kDepth > kRowDepth<kVec> ? kNormDeepThreads : kRowThreads<kVec>;
  static SmemGrant granted;
  const cudaError_t err = grant_smem(reinterpret_cast<const void*>(k),
                                     RowStream<kVec, kDepth>::bytes(most_threads), granted);
  if (err != cudaSuccess) return err;
  const int64_t most = (a.rows + p.rows - 1) / p.rows, full = row_ctas(p.threads, smem, sms);
  return launch_pdl(k, dim3(static_cast<unsigned>(most < full ? most : full)), dim3(p.threads), smem,
                    st, a);
}
template <class T>
cudaError_t launch_norm(const NormArgs& a, const RowPlan& p, int sms, cudaStream_t st) {
  // few rows of many items: twice as many on their way
  if (p.vec == 1 && p.rows == 1 && a.rows <= sms && p.threads <= kNormDeepThreads)
    return launch_norm<T, 1, 16, true>(a, p, sms, st);
  const bool one = p.rows == 1;  // (of at most two vectors a thread)
  switch (p.vec) {
    case 1: return one ? launch_norm<T, 1, kRowDepth<1>, true>(a, p, sms, st)
                       : launch_norm<T, 1, kRowDepth<1>, false>(a, p, sms, st);
    case 2: return one ? launch_norm<T, 2, kRowDepth<2>, true>(a, p, sms, st)
                       : launch_norm<T, 2, kRowDepth<2>, false>(a, p, sms, st);
    case 3: return launch_norm<T, 3, kRowDepth<3>, false>(a, p, sms, st);
    default: return launch_norm<T, 4, kRowDepth<4>, false>(a, p, sms, st);
  }
}
template <class T, int kVec, bool kOne, int kThreads = kRowThreads<kVec>>
cudaError_t launch_norm_grad(const NormGradArgs& a, const RowPlan& p, int ctas, cudaStream_t st) {
  auto* k = mrs_norm_grad_kernel<T, kVec, kOne, kThreads>;
  auto bytes = [](int threads) {  // the items, and 32 bytes of sums for each vector
    return RowStream<kVec, kRowDepth<kVec>>::bytes(threads) + static_cast<size_t>(32) * kVec * threads;
  };
  static SmemGrant granted;
  const cudaError_t err =
      grant_smem(reinterpret_cast<const void*>(k), bytes(kThreads), granted);
  if (err != cudaSuccess) return err;
  return launch_pdl(k, dim3(ctas), dim3(p.threads), bytes(p.threads), st, a);
}
template <class T>
cudaError_t launch_norm_grad(const NormGradArgs& a, const RowPlan& p, int ctas, cudaStream_t st) {
  const bool one = p.rows == 1;
  if (p.vec == 2 && one && p.threads <= kNormTwoThreads)
    return launch_norm_grad<T, 2, true, kNormTwoThreads>(a, p, ctas, st);
  switch (p.vec) {
    case 1: return one ? launch_norm_grad<T, 1, true>(a, p, ctas, st)
                       : launch_norm_grad<T, 1, false>(a, p, ctas, st);
    case 2: return one ? launch_norm_grad<T, 2, true>(a, p, ctas, st)
                       : launch_norm_grad<T, 2, false>(a, p, ctas, st);
    case 3: return launch_norm_grad<T, 3, false>(a, p, ctas, st);
    default: return launch_norm_grad<T, 4, false>(a, p, ctas, st);
  }
}

bool bad_row_cols(int cols) { return cols < 8 || cols > kRowMaxCols || cols % 8 != 0; }
bool bad_half(int dtype) { return dtype != MOE_RS_BF16 && dtype != MOE_RS_FP16; }
bool bad_gain(int gain_dtype, int dtype) {
  return gain_dtype != dtype && gain_dtype != MOE_RS_FP32;
}
// Rows that a launch and every offset hold.
bool too_many(int64_t rows, int64_t parts, int64_t stride) {
  return rows > INT32_MAX || parts * rows > (int64_t{1} << 40) || stride > (int64_t{1} << 31);
}

}  // namespace
}  // namespace mrs

using namespace mrs;

extern "C" {

int moe_rms_norm(const void* x, int dtype, int64_t x_stride, int parts, const void* residual,
                 int64_t residual_stride, int64_t rows, int cols, const void* gain, int gain_dtype,
                 float eps, void* y, void* sum, uint8_t* codes, float* scales, float* rstd,
                 cudaStream_t stream) {
  if (bad_half(dtype) || bad_gain(gain_dtype, dtype)) return MOE_RS_ERR_BAD_DTYPE;
  if (rows < 0) return MOE_RS_ERR_BAD_ROWS;
  if (parts < 1 || parts > kMaxTopk) return MOE_RS_ERR_BAD_TOPK;
  if (bad_row_cols(cols) || x_stride < cols || (residual && residual_stride < cols))
    return MOE_RS_ERR_BAD_COLS;
  if (!(eps >= 0.0f) || eps > 1.0f) return MOE_RS_ERR_BAD_SCALE;
  if (too_many(rows, parts, x_stride) || (residual && residual_stride > (int64_t{1} << 31)))
    return MOE_RS_ERR_OVERFLOW;
  if (rows == 0) return MOE_RS_OK;
  if (!x || !gain || (!y && !sum && !codes && !rstd) || (codes == nullptr) != (scales == nullptr))
    return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(x, 16) || x_stride % 8 != 0 || !aligned(residual, 16) ||
      (residual && residual_stride % 8 != 0) || !aligned(gain, 16) || !aligned(y, 16) ||
      !aligned(sum, 16) || !aligned(codes, 8) || !aligned(scales, 4) || !aligned(rstd, 4))
    return MOE_RS_ERR_MISALIGNED;
  const size_t n = static_cast<size_t>(rows) * cols;
  const size_t c = static_cast<size_t>(cols);
  // the residual stream may be updated in place
  const bool in_place = sum != nullptr && sum == residual && residual_stride == cols;
  const Span outs[] = {span(y, y ? 2 * n : 0), span(sum, sum ? 2 * n : 0),
                       span(codes, codes ? n : 0), span(scales, scales ? 4 * rows : 0),
                       span(rstd, rstd ? 4 * rows : 0)};
  const Span ins[] = {rows_span(x, rows * parts, cols, x_stride, 2),
                      span(gain, c * (gain_dtype == MOE_RS_FP32 ? 4 : 2)),
                      rows_span(in_place ? nullptr : residual, rows, cols, residual_stride, 2)};
  if (any_alias(outs, 5, ins, 3)) return MOE_RS_ERR_ALIAS;
  const int sms = sm_count();
  if (sms == 0) return launch_status(cudaErrorInvalidDevice);
  // Two vectors a thread halve the instructions of an item (8192 x 3584: 60 us with one, 52 with two,
  // before the gain stayed in registers);
  // few rows are spread over more threads (one token of 16 rows 8.9 and 10.9).
  const RowPlan p = row_plan(cols, rows <= sms ? 1 : 2);
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.gain = gain;
  a.x_stride = static_cast<size_t>(x_stride);
  a.residual_stride = static_cast<size_t>(residual_stride);
  a.rows = rows;
  a.parts = parts;
  a.vecs = cols / 8;
  a.tpr = p.tpr;
  a.per_cta = p.rows;
  a.gain_f32 = gain_dtype == MOE_RS_FP32;
  a.eps = eps;
  a.inv_cols = 1.0f / static_cast<float>(cols);
  a.y = y;
  a.sum = sum;
  a.codes = codes;
  a.scales = scales;
  a.rstd = rstd;
  return launch_status(dtype == MOE_RS_BF16 ? launch_norm<__nv_bfloat16>(a, p, sms, stream)
                                            : launch_norm<__half>(a, p, sms, stream));
}

size_t moe_rms_norm_backward_workspace_bytes(int cols) {
  if (bad_row_cols(cols)) return 0;
  const RowPlan p = norm_grad_plan(cols);
  return static_cast<size_t>(norm_grad_ctas(p, kNormMaxSms)) * p.rows * cols * 4;
}

int moe_rms_norm_backward(const void* s, int dtype, const void* gain, int gain_dtype,
                          const float* rstd, const void* grad, const void* grad_rows, int parts,
                          const void* grad_sum, int64_t rows, int cols, void* grad_x,
                          float* grad_gain, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  if (bad_half(dtype) || bad_gain(gain_dtype, dtype)) return MOE_RS_ERR_BAD_DTYPE;
  if (rows < 0) return MOE_RS_ERR_BAD_ROWS;
  if (parts < 1 || parts > kMaxTopk) return MOE_RS_ERR_BAD_TOPK;
  if (bad_row_cols(cols)) return MOE_RS_ERR_BAD_COLS;
  if (too_many(rows, parts, cols)) return MOE_RS_ERR_OVERFLOW;
  const size_t need = moe_rms_norm_backward_workspace_bytes(cols);
  if (grad_gain && (!workspace || workspace_bytes < need)) return MOE_RS_ERR_WORKSPACE;
  if (rows > 0 && (!s || !gain || !rstd || !grad_x || (!grad && !grad_rows)))
    return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(s, 16) || !aligned(gain, 16) || !aligned(rstd, 4) || !aligned(grad, 16) ||
      !aligned(grad_rows, 16) || !aligned(grad_sum, 16) || !aligned(grad_x, 16) ||
      !aligned(grad_gain, 4) || !aligned(workspace, 16))
    return MOE_RS_ERR_MISALIGNED;
  const size_t n = 2 * static_cast<size_t>(rows) * cols, c = static_cast<size_t>(cols);
  const Span outs[] = {span(grad_x, n), span(grad_gain, grad_gain ? 4 * c : 0),
                       span(workspace, grad_gain ? workspace_bytes : 0)};
  const Span ins[] = {span(s, n), span(gain, c * (gain_dtype == MOE_RS_FP32 ? 4 : 2)),
                      span(rstd, 4 * static_cast<size_t>(rows)), span(grad, grad ? n : 0),
                      span(grad_rows, grad_rows ? n * parts : 0), span(grad_sum, grad_sum ? n : 0)};
  if (any_alias(outs, 3, ins, 6)) return MOE_RS_ERR_ALIAS;
  if (rows == 0 && !grad_gain) return MOE_RS_OK;
  const int sms = sm_count();
  if (sms == 0) return launch_status(cudaErrorInvalidDevice);
  const RowPlan p = norm_grad_plan(cols);
  NormGradArgs a{};
  a.s = s;
  a.gain = gain;
  a.grad = grad;
  a.grad_rows = grad_rows;
  a.grad_sum = grad_sum;
  a.rstd = rstd;
  a.rows = rows;
  a.parts = parts;
  a.vecs = cols / 8;
  a.tpr = p.tpr;
  a.per_cta = p.rows;
  a.gain_f32 = gain_dtype == MOE_RS_FP32;
  a.inv_cols = 1.0f / static_cast<float>(cols);
  a.grad_x = grad_x;
  a.partial = grad_gain ? static_cast<float*>(workspace) : nullptr;
  // without rows one CTA leaves the zeros that the sums are made of
  const int64_t most = rows == 0 ? 1 : (rows + p.rows - 1) / p.rows;
  const int full = norm_grad_ctas(p, sms < kNormMaxSms ? sms : kNormMaxSms);
  const int ctas = most < full ? static_cast<int>(most) : full;
  cudaError_t err = dtype == MOE_RS_BF16 ? launch_norm_grad<__nv_bfloat16>(a, p, ctas, stream)
                                         : launch_norm_grad<__half>(a, p, ctas, stream);
  if (err == cudaSuccess && grad_gain)
    err = launch_pdl(mrs_norm_gain_kernel, dim3((cols + 31) / 32), dim3(256), 0, stream,
                     static_cast<const float*>(a.partial), ctas * p.rows, cols, grad_gain);
  return launch_status(err);
}

}  // extern "C"
