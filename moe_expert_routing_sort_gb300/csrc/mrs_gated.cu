// mrs_gated.cu -- the gated activation between two experts' products, its gradient, and rows to
// 8 bits.
//
// Per row r, over c < cols, a = x[r, c], b = x[r, cols + c], w = weights[r] (1 without weights):
//   y[r, c] = w * a * sig(a) * b                        to 16 bits, or to e4m3 with the row's scale
// and its gradient, d = grad[r, c]:
//   grad_a = w d b sig(a) (1 + a (1 - sig(a))),   grad_b = w d a sig(a)
//   grad_w = sum over c of d a sig(a) b
// All in fp32, one rounding at the end.  The routing weight belongs here in training: the second
// product is then a plain one, and its gradients need no weights.  1 - sig(a) is sig(-a), which
// keeps its bits where sig(a) is next to 1.
//
// Bound by memory: one read of every input, one write of every output, a row in registers (the
// activation's with two vectors a thread all but 24 bytes of each thread); a thread's next vectors are on
// their way while it computes.  131072 x 384 46 us and the gradient of 65536 x 2048 199 us, 97 and 99 %
// of the rate of a copy.  In 8 bits 131072 x 384 51 us, of 37: a row's two meetings with its scale.  Rows
// to 8 bits: 131072 x 7168 in fp32 653 us, of 692, 688128 x 3584 in bf16 1388, of 1090.
#include "mrs_rows.cuh"

namespace mrs {

struct GatedArgs {
  const void* x;
  const void* grad;       // of the gradient: [rows, cols]
  const float* weights;   // or null
  size_t x_stride;
  int64_t rows;
  int vecs, tpr, per_cta;
  void* y;                // [rows, cols]; of the gradient [rows, 2 cols]
  unsigned char* codes;
  float* scales;
  float* grad_weights;    // or null
};

// sig(a) as up * root, and sig(-a).  Of a negative a, root is exp(a / 2) and up has it once more: far
// below zero sig(a) is smaller than any fp32 number while its product with a large b, or a large
// gradient, is not, so that its second half is multiplied behind them.  root is zero below a = -174,
// where no such product reaches 2^-124.  (__expf keeps subnormal results, and its scaling for them
// costs more than these multiplications: gradient of 65536 x 2048 205 us with it.)
__device__ __forceinline__ void sigmoids(float a, float& up, float& root, float& down) {
  float half, big;  // half in [0, 1]
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(half) : "f"(-0.72134752f * fabsf(a)));  // log2(e) / 2
  const float e = half * half;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(big) : "f"(1.0f + e));
  root = a >= 0.0f ? 1.0f : half;
  up = big * root;
  down = a >= 0.0f ? e * big : big;
}

// What a thread takes of a row, on its way while the row before is computed.
template <int kVec>
struct GatedRow {
  uint4 a[kVec], b[kVec];
  float w;
};

template <class T, int kVec>
__global__ void __launch_bounds__(kRowThreads<kVec>) mrs_gated_kernel(const GatedArgs a) {
  __shared__ RowTotals meet[32];
  pdl_trigger();
  const int tid = threadIdx.x, in_cta = tid / a.tpr, place = tid - in_cta * a.tpr;
  const int64_t step = static_cast<int64_t>(gridDim.x) * a.per_cta;
  const size_t cols = 8 * static_cast<size_t>(a.vecs);
  auto load = [&](int64_t row, GatedRow<kVec>& r) {
    if (row >= a.rows) return;
    r.w = a.weights != nullptr ? __ldg(a.weights + row) : 1.0f;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int at = i * a.tpr + place;
      if (at >= a.vecs) continue;
      r.a[i] = load8<T>(x, 8 * static_cast<size_t>(at));
      r.b[i] = load8<T>(x, cols + 8 * at);
    }
  };
  pdl_wait();
  int64_t row = static_cast<int64_t>(blockIdx.x) * a.per_cta + in_cta;
  GatedRow<kVec> now, next;
  load(row, now);
  // (the rows of a CTA take the same number of turns: they meet in the reduction)
  for (; row - in_cta < a.rows; row += step, now = next) {
    const bool live = row < a.rows;
    load(row + step, next);
    float v[kVec][8];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int at = i * a.tpr + place;
      if (!live || at >= a.vecs) continue;
      float b[8];
      unpack8<T>(now.a[i], v[i]);
      unpack8<T>(now.b[i], b);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float up, root, down;
        sigmoids(v[i][k], up, root, down);
        v[i][k] = now.w * (v[i][k] * up * b[k] * root);
      }
      if (a.y != nullptr)
        *reinterpret_cast<uint4*>(static_cast<T*>(a.y) + row * cols + 8 * at) = pack8<T>(v[i]);
      if (a.codes != nullptr) {
#pragma unroll
        for (int k = 0; k < 8; ++k) top = larger(top, v[i][k]);
      }
    }
    if (a.codes == nullptr) continue;
    const float scale = fp8_scale(row_totals(0.0f, __float_as_uint(top), a.tpr, meet).top);
    if (!live) continue;
    if (place == 0) a.scales[row] = scale;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int at = i * a.tpr + place;
      if (at < a.vecs)
        *reinterpret_cast<uint2*>(a.codes + row * cols + 8 * at) = fp8_codes_of(v[i], scale);
    }
  }
}

template <class T, int kVec>
__global__ void __launch_bounds__(kRowThreads<kVec>) mrs_gated_grad_kernel(const GatedArgs a) {
  __shared__ RowTotals meet[32];
  pdl_trigger();
  const int tid = threadIdx.x, in_cta = tid / a.tpr, place = tid - in_cta * a.tpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * a.per_cta + in_cta;
  const bool live = row < a.rows;
  const size_t cols = 8 * static_cast<size_t>(a.vecs);
  pdl_wait();
  const float w = live && a.weights != nullptr ? __ldg(a.weights + row) : 1.0f;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  T* out = static_cast<T*>(a.y) + row * 2 * cols;
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int at = i * a.tpr + place;
    if (!live || at >= a.vecs) continue;
    float g[8], b[8], d[8], ga[8], gb[8];
    unpack8<T>(load8<T>(x, 8 * static_cast<size_t>(at)), g);
    unpack8<T>(load8<T>(x, cols + 8 * at), b);
    unpack8<T>(load8<T>(a.grad, row * cols + 8 * at), d);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float up, root, down;
      sigmoids(g[k], up, root, down);
      const float act = g[k] * up, wd = w * d[k];
      dot += d[k] * act * b[k] * root;
      ga[k] = wd * b[k] * (up * (1.0f + g[k] * down)) * root;
      gb[k] = wd * act * root;
    }
    *reinterpret_cast<uint4*>(out + 8 * at) = pack8<T>(ga);
    *reinterpret_cast<uint4*>(out + cols + 8 * at) = pack8<T>(gb);
  }
  if (a.grad_weights == nullptr) return;
  const float sum = row_totals(dot, 0u, a.tpr, meet).sum;
  if (live && place == 0) a.grad_weights[row] = sum;
}

// Rows of bf16, fp16 or fp32 to 8 bits.
template <class T, int kVec>
__global__ void __launch_bounds__(kRowThreads<kVec>) mrs_fp8_quantize_kernel(const GatedArgs a) {
  __shared__ RowTotals meet[32];
  pdl_trigger();
  const int tid = threadIdx.x, in_cta = tid / a.tpr, place = tid - in_cta * a.tpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * a.per_cta + in_cta;
  const bool live = row < a.rows;
  const size_t cols = 8 * static_cast<size_t>(a.vecs);
  pdl_wait();
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  float v[kVec][8];
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int at = i * a.tpr + place;
    if (!live || at >= a.vecs) continue;
    if constexpr (sizeof(T) == 4)
      load_columns<__half>(x, true, at, v[i]);
    else
      unpack8<T>(load8<T>(x, 8 * static_cast<size_t>(at)), v[i]);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = larger(top, v[i][k]);
  }
  const float scale = fp8_scale(row_totals(0.0f, __float_as_uint(top), a.tpr, meet).top);
  if (!live) return;
  if (place == 0) a.scales[row] = scale;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int at = i * a.tpr + place;
    if (at < a.vecs)
      *reinterpret_cast<uint2*>(a.codes + row * cols + 8 * at) = fp8_codes_of(v[i], scale);
  }
}

namespace {

// Rows up to which a row is spread over as many threads as it has vectors; more take two vectors a thread.
// us in a graph with one and with two: activation and gradient of 16 rows of 2048 1.27 1.62 and 1.63 2.17,
// of 152 rows 1.37 1.76 and 1.78 2.25, of 608 rows of 8192 4.5 4.7 and 10.0 7.3 (to 8 bits 7.1 6.2), of 304
// rows 2.9 2.9 and 5.2 4.2.
constexpr int64_t kGatedFewRows = 152;

enum class GatedKind { kForward, kGradient, kQuantize };

template <class T, int kVec, GatedKind kKind>
auto* gated_kernel() {
  if constexpr (kKind == GatedKind::kForward) return mrs_gated_kernel<T, kVec>;
  else if constexpr (kKind == GatedKind::kGradient) return mrs_gated_grad_kernel<T, kVec>;
  else return mrs_fp8_quantize_kernel<T, kVec>;
}

template <class T, int kVec, GatedKind kKind>
cudaError_t launch_gated(const GatedArgs& a, const RowPlan& p, int sms, cudaStream_t st) {
  auto* k = gated_kernel<T, kVec, kKind>();
  const int64_t most = (a.rows + p.rows - 1) / p.rows;
  // The activation's CTAs go round (131072 x 384: 46 us, and 54 with a CTA for every 16 rows); the
  // gradient's do not (65536 x 2048: 196 us, and 224 so: its next row takes registers that its CTAs
  // have no room for).
  const int64_t full = kKind == GatedKind::kForward ? row_ctas(p.threads, 0, sms) : most;
  return launch_pdl(k, dim3(static_cast<unsigned>(most < full ? most : full)), dim3(p.threads), 0, st,
                    a);
}
template <class T, GatedKind kKind>
cudaError_t launch_gated(const GatedArgs& a, const RowPlan& p, cudaStream_t st) {
  const int sms = sm_count();
  if (sms == 0) return cudaErrorInvalidDevice;
  switch (p.vec) {
    case 1: return launch_gated<T, 1, kKind>(a, p, sms, st);
    case 2: return launch_gated<T, 2, kKind>(a, p, sms, st);
    case 3: return launch_gated<T, 3, kKind>(a, p, sms, st);
    default: return launch_gated<T, 4, kKind>(a, p, sms, st);
  }
}

// Checks of `rows` rows of `width` elements of `size` bytes, `stride` elements apart.
int check_gated(const void* x, int64_t x_stride, int64_t rows, int cols, int width, size_t size) {
  if (rows < 0) return MOE_RS_ERR_BAD_ROWS;
  if (cols < 8 || cols > kRowMaxCols || cols % 8 != 0 || x_stride < width)
    return MOE_RS_ERR_BAD_COLS;
  if (rows > INT32_MAX || x_stride > (int64_t{1} << 31)) return MOE_RS_ERR_OVERFLOW;
  if (rows == 0) return MOE_RS_OK;
  if (!x) return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(x, 16) || static_cast<size_t>(x_stride) * size % 16 != 0)
    return MOE_RS_ERR_MISALIGNED;
  return MOE_RS_OK;
}

GatedArgs gated_args(const void* x, int64_t x_stride, int64_t rows, int cols, const RowPlan& p) {
  GatedArgs a{};
  a.x = x;
  a.x_stride = static_cast<size_t>(x_stride);
  a.rows = rows;
  a.vecs = cols / 8;
  a.tpr = p.tpr;
  a.per_cta = p.rows;
  return a;
}

}  // namespace
}  // namespace mrs

using namespace mrs;

extern "C" {

int moe_swiglu(const void* x, int dtype, int64_t x_stride, int64_t rows, int cols,
               const float* weights, void* y, uint8_t* codes, float* scales, cudaStream_t stream) {
  if (dtype != MOE_RS_BF16 && dtype != MOE_RS_FP16) return MOE_RS_ERR_BAD_DTYPE;
  const int rc = check_gated(x, x_stride, rows, cols, 2 * cols, 2);
  if (rc || rows == 0) return rc;
  if ((!y && !codes) || (codes == nullptr) != (scales == nullptr)) return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(weights, 4) || !aligned(y, 16) || !aligned(codes, 8) || !aligned(scales, 4))
    return MOE_RS_ERR_MISALIGNED;
  const size_t n = static_cast<size_t>(rows) * cols, r = static_cast<size_t>(rows);
  const Span outs[] = {span(y, y ? 2 * n : 0), span(codes, codes ? n : 0),
                       span(scales, scales ? 4 * r : 0)};
  const Span ins[] = {rows_span(x, rows, 2 * cols, x_stride, 2), span(weights, weights ? 4 * r : 0)};
  if (any_alias(outs, 3, ins, 2)) return MOE_RS_ERR_ALIAS;
  const RowPlan p = row_plan(cols, rows <= kGatedFewRows ? 1 : 2);
  GatedArgs a = gated_args(x, x_stride, rows, cols, p);
  a.weights = weights;
  a.y = y;
  a.codes = codes;
  a.scales = scales;
  return launch_status(dtype == MOE_RS_BF16
                           ? launch_gated<__nv_bfloat16, GatedKind::kForward>(a, p, stream)
                           : launch_gated<__half, GatedKind::kForward>(a, p, stream));
}

int moe_swiglu_backward(const void* grad, const void* x, int dtype, int64_t x_stride, int64_t rows,
                        int cols, const float* weights, void* grad_x, float* grad_weights,
                        cudaStream_t stream) {
  if (dtype != MOE_RS_BF16 && dtype != MOE_RS_FP16) return MOE_RS_ERR_BAD_DTYPE;
  const int rc = check_gated(x, x_stride, rows, cols, 2 * cols, 2);
  if (rc || rows == 0) return rc;
  if (!grad || !grad_x) return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(grad, 16) || !aligned(weights, 4) || !aligned(grad_x, 16) ||
      !aligned(grad_weights, 4))
    return MOE_RS_ERR_MISALIGNED;
  const size_t n = static_cast<size_t>(rows) * cols, r = static_cast<size_t>(rows);
  const Span outs[] = {span(grad_x, 4 * n), span(grad_weights, grad_weights ? 4 * r : 0)};
  const Span ins[] = {span(grad, 2 * n), rows_span(x, rows, 2 * cols, x_stride, 2),
                      span(weights, weights ? 4 * r : 0)};
  if (any_alias(outs, 2, ins, 3)) return MOE_RS_ERR_ALIAS;
  const RowPlan p = row_plan(cols, rows <= kGatedFewRows ? 1 : 2);
  GatedArgs a = gated_args(x, x_stride, rows, cols, p);
  a.grad = grad;
  a.weights = weights;
  a.y = grad_x;
  a.grad_weights = grad_weights;
  return launch_status(dtype == MOE_RS_BF16
                           ? launch_gated<__nv_bfloat16, GatedKind::kGradient>(a, p, stream)
                           : launch_gated<__half, GatedKind::kGradient>(a, p, stream));
}

int moe_fp8_quantize(const void* x, int x_dtype, int64_t rows, int cols, int64_t x_stride,
                     uint8_t* codes, float* scales, cudaStream_t stream) {
  if (x_dtype != MOE_RS_BF16 && x_dtype != MOE_RS_FP16 && x_dtype != MOE_RS_FP32)
    return MOE_RS_ERR_BAD_DTYPE;
  const size_t size = x_dtype == MOE_RS_FP32 ? 4 : 2;
  const int rc = check_gated(x, x_stride, rows, cols, cols, size);
  if (rc || rows == 0) return rc;
  if (!codes || !scales) return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(codes, 8) || !aligned(scales, 4)) return MOE_RS_ERR_MISALIGNED;
  const Span outs[] = {span(codes, static_cast<size_t>(rows) * cols),
                       span(scales, 4 * static_cast<size_t>(rows))};
  const Span ins[] = {rows_span(x, rows, cols, x_stride, size)};
  if (any_alias(outs, 2, ins, 1)) return MOE_RS_ERR_ALIAS;
  const RowPlan p = row_plan(cols, rows <= kGatedFewRows ? 1 : 2);
  GatedArgs a = gated_args(x, x_stride, rows, cols, p);
  a.codes = codes;
  a.scales = scales;
  return launch_status(x_dtype == MOE_RS_FP32 ? launch_gated<float, GatedKind::kQuantize>(a, p, stream)
                       : x_dtype == MOE_RS_FP16
                           ? launch_gated<__half, GatedKind::kQuantize>(a, p, stream)
                           : launch_gated<__nv_bfloat16, GatedKind::kQuantize>(a, p, stream));
}

}  // extern "C"
