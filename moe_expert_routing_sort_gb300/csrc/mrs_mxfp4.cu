// mrs_mxfp4.cu -- rows to microscaled 4-bit floating point (MXFP4) and back.
//
// 32 consecutive elements of a row share one power-of-two scale 2^e, stored as the byte
// e + 127 (E8M0); each element is stored as the nearest of {0, 1/2, 1, 3/2, 2, 3, 4, 6} * 2^e
// with a sign (E2M1), two per byte, the lower column in the low nibble.  Per block of 32:
//   e     = floor(log2(max |x|)) - 2, clamped to [-127, 125]: the largest magnitude lands in
//           [4, 8), so the codes' top binade [4, 6] is used and what is beyond 6 saturates
//   code  = nearest of x * 2^-e, ties to the even code, at most 6 in magnitude
// x * 2^-e is exact (a power of two, and fp32 holds every input type), so the conversion
// instruction's single rounding is the only one.  A block of zeros (and one whose maximum is
// below 2^-125) takes the smallest scale byte, 0.  A block holding an infinity or a NaN takes
// the scale byte 255 (the format's NaN) with zero codes: it reads back as NaN, so a non-finite
// value is never turned into a finite one.
// Bound: one read of the input and one write of half a byte per element plus a scale byte per
// 32.  A thread takes 8 consecutive elements (one 16-byte load of a 16-bit type), the four
// threads of a block agree on the maximum with two shuffles, and a warp writes 128 contiguous
// bytes of codes.  A thread has four such units, a CTA's width apart, all loaded before the first
// is used (one unit a thread: 8192 x 3584 in 20.9 us, and 17.3 back).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mrs_args.h"
#include "mrs_internal.h"
#include "mrs_mx.cuh"

namespace mrs {

constexpr int kMxThreads = 256;
constexpr int kMxUnits = 4;  // units of 8 elements per thread

struct MxQuantArgs {
  const void* x;
  size_t units;      // rows * cols / 8
  unsigned upr;      // units of 8 elements per row
  size_t stride;     // elements between rows of x
  unsigned scols;    // scale bytes per row (a multiple of 4)
  unsigned char* codes;
  unsigned char* scales;
};

struct MxDequantArgs {
  const unsigned char* codes;
  const unsigned char* scales;
  size_t units;
  unsigned upr;
  size_t stride;  // elements between rows of y
  unsigned scols;
  void* y;
};

// Eight consecutive elements as fp32.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = *reinterpret_cast<const __half2*>(&w[i]);
    const float2 f = __half22float2(h);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// Where unit `u` lies: its row, and its place in the row.
struct MxUnit {
  size_t row;
  unsigned c;
  bool in;
};
// The thread's units.  The division is done once; the others are a CTA's width further.
__device__ __forceinline__ void mx_units(size_t units, unsigned upr, MxUnit (&at)[kMxUnits]) {
  size_t u = static_cast<size_t>(blockIdx.x) * (kMxThreads * kMxUnits) + threadIdx.x;
  size_t row = u < units ? u / upr : 0;
  unsigned c = static_cast<unsigned>(u - row * upr);
  if (u >= units) c = 0;
#pragma unroll
  for (int j = 0; j < kMxUnits; ++j) {
    at[j] = MxUnit{row, c, u < units};
    u += kMxThreads;
    c += kMxThreads;
    if (c >= upr) {  // (32 bits: cheap)
      row += c / upr;
      c %= upr;
    }
  }
}

template <class In>
__global__ void __launch_bounds__(kMxThreads) mrs_mxfp4_quantize_kernel(const MxQuantArgs a) {
  pdl_trigger();
  MxUnit at[kMxUnits];
  mx_units(a.units, a.upr, at);
  pdl_wait();
  float v[kMxUnits][8];
#pragma unroll
  for (int j = 0; j < kMxUnits; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
    // the four threads of a block are all in or all out (a row holds a multiple of four units)
    if (at[j].in)
      load8(static_cast<const In*>(a.x) + at[j].row * a.stride + 8 * static_cast<size_t>(at[j].c),
            v[j]);
  }
#pragma unroll
  for (int j = 0; j < kMxUnits; ++j) {
    uint32_t top = 0u;  // bits of the largest magnitude (ordered like the magnitudes)
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[j][i]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
    if (at[j].in) {
      const uint32_t ef = top >> 23;  // exponent field; 0 (zero, subnormal) clamps like 1 does
      uint32_t scale = ef > 2u ? ef - 2u : 0u;
      uint32_t code = 0u;
      if (ef == 255u) {
        scale = 255u;
      } else {
        const float inv = __uint_as_float((254u - scale) << 23);  // 2^(127 - scale), normal
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] *= inv;
        code = e2m1x8(v[j]);
      }
      const size_t row = at[j].row;
      const unsigned c = at[j].c;
      *reinterpret_cast<uint32_t*>(a.codes + row * (4 * static_cast<size_t>(a.upr)) +
                                   4 * static_cast<size_t>(c)) = code;
      if ((c & 3u) == 0u) {
        unsigned char* s = a.scales + row * a.scols;
        s[c >> 2] = static_cast<unsigned char>(scale);
        if (c + 4u == a.upr)  // the row's last block also clears the padding bytes
          for (unsigned p = (c >> 2) + 1u; p < a.scols; ++p) s[p] = 0;
      }
    }
    __syncwarp();
  }
}

template <class Out>
__global__ void __launch_bounds__(kMxThreads) mrs_mxfp4_dequantize_kernel(const MxDequantArgs a) {
  pdl_trigger();
  MxUnit at[kMxUnits];
  mx_units(a.units, a.upr, at);
  pdl_wait();
  uint32_t code[kMxUnits], scale[kMxUnits];
#pragma unroll
  for (int j = 0; j < kMxUnits; ++j) {
    code[j] = scale[j] = 0u;
    if (!at[j].in) continue;
    code[j] = __ldg(reinterpret_cast<const uint32_t*>(a.codes) +
                    at[j].row * static_cast<size_t>(a.upr) + at[j].c);
    scale[j] = __ldg(a.scales + at[j].row * a.scols + (at[j].c >> 2));
  }
#pragma unroll
  for (int j = 0; j < kMxUnits; ++j) {
    if (!at[j].in) continue;
    float v[8];
    e2m1_values(code[j], v);
    const float s = e8m0_value(scale[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s;
    Out* y = static_cast<Out*>(a.y) + at[j].row * a.stride + 8 * static_cast<size_t>(at[j].c);
    if constexpr (sizeof(Out) == 4) {
      reinterpret_cast<float4*>(y)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(y)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      // the one rounding of this direction: exact in bf16 down to its smallest subnormal
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(y) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

}  // namespace mrs

// ------------------------------------------------------------------------- entry points
using namespace mrs;

namespace {

bool bad_cols(int cols) { return cols < 32 || cols > MOE_RS_MXFP4_MAX_COLS || cols % 32 != 0; }

// Rows of `cols` elements of `size` bytes, `stride` elements apart.
size_t row_span(int64_t rows, int cols, int64_t stride, size_t size) {
  return rows == 0 ? 0
                   : (static_cast<size_t>(rows - 1) * static_cast<size_t>(stride) +
                      static_cast<size_t>(cols)) * size;
}

int check_rows(const void* x, int64_t rows, int cols, int64_t stride, size_t size) {
  if (rows < 0) return MOE_RS_ERR_BAD_ROWS;
  if (bad_cols(cols)) return MOE_RS_ERR_BAD_COLS;
  if (stride < cols) return MOE_RS_ERR_BAD_COLS;
  // blocks of the launch: one per 256 threads of 8 elements
  if (rows > (int64_t{1} << 40) || stride > (int64_t{1} << 40) || rows * (cols / 8) > (int64_t{INT32_MAX} * kMxThreads))
    return MOE_RS_ERR_OVERFLOW;
  if (rows == 0) return MOE_RS_OK;
  if (!x) return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(x, 16) || (static_cast<size_t>(stride) * size) % 16 != 0)
    return MOE_RS_ERR_MISALIGNED;
  return MOE_RS_OK;
}

}  // namespace

extern "C" {

int moe_mxfp4_scale_cols(int cols) { return bad_cols(cols) ? 0 : (cols + 127) / 128 * 4; }

int moe_mxfp4_quantize(const void* x, int x_dtype, int64_t rows, int cols, int64_t x_stride,
                       uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
  if (x_dtype != MOE_RS_BF16 && x_dtype != MOE_RS_FP16 && x_dtype != MOE_RS_FP32)
    return MOE_RS_ERR_BAD_DTYPE;
  const size_t size = x_dtype == MOE_RS_FP32 ? 4 : 2;
  const int rc = check_rows(x, rows, cols, x_stride, size);
  if (rc || rows == 0) return rc;
  if (!codes || !scales) return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(codes, 16) || !aligned(scales, 4)) return MOE_RS_ERR_MISALIGNED;
  const int scols = moe_mxfp4_scale_cols(cols);
  const Span outs[] = {span(codes, static_cast<size_t>(rows) * (cols / 2)),
                       span(scales, static_cast<size_t>(rows) * scols)};
  const Span ins[] = {span(x, row_span(rows, cols, x_stride, size))};
  if (any_alias(outs, 2, ins, 1)) return MOE_RS_ERR_ALIAS;
  MxQuantArgs a{};
  a.x = x;
  a.upr = static_cast<unsigned>(cols / 8);
  a.units = static_cast<size_t>(rows) * a.upr;
  a.stride = static_cast<size_t>(x_stride);
  a.scols = static_cast<unsigned>(scols);
  a.codes = codes;
  a.scales = scales;
  const dim3 grid(static_cast<unsigned>((a.units + kMxThreads * kMxUnits - 1) / (kMxThreads * kMxUnits)));
  auto* k = x_dtype == MOE_RS_FP32   ? mrs_mxfp4_quantize_kernel<float>
            : x_dtype == MOE_RS_FP16 ? mrs_mxfp4_quantize_kernel<__half>
                                     : mrs_mxfp4_quantize_kernel<__nv_bfloat16>;
  return launch_status(launch_pdl(k, grid, dim3(kMxThreads), 0, stream, a));
}

int moe_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols,
                         void* y, int y_dtype, int64_t y_stride, cudaStream_t stream) {
  if (y_dtype != MOE_RS_BF16 && y_dtype != MOE_RS_FP32) return MOE_RS_ERR_BAD_DTYPE;
  const size_t size = y_dtype == MOE_RS_FP32 ? 4 : 2;
  const int rc = check_rows(y, rows, cols, y_stride, size);
  if (rc || rows == 0) return rc;
  if (!codes || !scales) return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(codes, 16) || !aligned(scales, 4)) return MOE_RS_ERR_MISALIGNED;
  const int scols = moe_mxfp4_scale_cols(cols);
  const Span outs[] = {span(y, row_span(rows, cols, y_stride, size))};
  const Span ins[] = {span(codes, static_cast<size_t>(rows) * (cols / 2)),
                      span(scales, static_cast<size_t>(rows) * scols)};
  if (any_alias(outs, 1, ins, 2)) return MOE_RS_ERR_ALIAS;
  MxDequantArgs a{};
  a.codes = codes;
  a.scales = scales;
  a.upr = static_cast<unsigned>(cols / 8);
  a.units = static_cast<size_t>(rows) * a.upr;
  a.stride = static_cast<size_t>(y_stride);
  a.scols = static_cast<unsigned>(scols);
  a.y = y;
  const dim3 grid(static_cast<unsigned>((a.units + kMxThreads * kMxUnits - 1) / (kMxThreads * kMxUnits)));
  auto* k = y_dtype == MOE_RS_FP32 ? mrs_mxfp4_dequantize_kernel<float>
                                   : mrs_mxfp4_dequantize_kernel<__nv_bfloat16>;
  return launch_status(launch_pdl(k, grid, dim3(kMxThreads), 0, stream, a));
}

}  // extern "C"
