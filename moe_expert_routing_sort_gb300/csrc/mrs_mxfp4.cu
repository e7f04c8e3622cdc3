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
// 32.  A thread takes one block: 64 bytes of a 16-bit type in 32-byte loads (whole sectors), its
// maximum over packed pairs, one 16-byte store of codes and a scale byte beside its neighbours'.
// (Four threads a block, each four times 8 elements: 20.7 us for 8192 x 3584 and 13.1 back.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mrs_args.h"
#include "mrs_internal.h"
#include "mrs_mx.cuh"

namespace mrs {

constexpr int kMxThreads = 256;

struct MxQuantArgs {
  const void* x;
  size_t blocks;   // rows * cols / 32
  unsigned bpr;    // blocks per row
  size_t stride;   // elements between rows of x
  unsigned scols;  // scale bytes per row (a multiple of 4)
  int wide;        // rows start on 32 bytes
  unsigned char* codes;
  unsigned char* scales;
};

struct MxDequantArgs {
  const unsigned char* codes;
  const unsigned char* scales;
  size_t blocks;
  unsigned bpr;
  size_t stride;  // elements between rows of y
  unsigned scols;
  int wide;
  void* y;
};

// 32 bytes, as one access where the address allows it.
__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t* w) {
  if (wide) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldg(static_cast<const uint4*>(p)), b = __ldg(static_cast<const uint4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t* w) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// The largest magnitude of a block as fp32 bits, and its elements 8 j .. 8 j + 7 as fp32.  Bits
// without the sign are ordered like the magnitudes, infinities and NaN on top.
struct BlockFp32 {
  static constexpr int kWords = 32;
  uint32_t w[kWords];
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i) t = max(t, w[i] & 0x7fffffffu);
    return t;
  }
  __device__ __forceinline__ void eight(int j, float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[8 * j + i]);
  }
};
template <bool kBf16>
struct BlockHalf {
  static constexpr int kWords = 16;
  uint32_t w[kWords];
  static __device__ __forceinline__ float2 pair(uint32_t h) {
    if constexpr (kBf16) return make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&h));
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) t = __vmaxu2(t, w[i] & 0x7fff7fffu);
    const uint32_t m = max(t & 0xffffu, t >> 16);
    return __float_as_uint(pair(m).x);
  }
  __device__ __forceinline__ void eight(int j, float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = pair(w[4 * j + i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};

template <class Block>
__global__ void __launch_bounds__(kMxThreads) mrs_mxfp4_quantize_kernel(const MxQuantArgs a) {
  pdl_trigger();
  const size_t u = static_cast<size_t>(blockIdx.x) * kMxThreads + threadIdx.x;
  const size_t row = u / a.bpr;
  const unsigned c = static_cast<unsigned>(u - row * a.bpr);
  pdl_wait();
  if (u >= a.blocks) return;
  constexpr size_t kSize = Block::kWords / 8;  // bytes of an element
  const unsigned char* x =
      static_cast<const unsigned char*>(a.x) + (row * a.stride + 32 * static_cast<size_t>(c)) * kSize;
  Block b;
#pragma unroll
  for (int i = 0; i < Block::kWords; i += 8) load32(x + 4 * i, a.wide != 0, b.w + i);
  const uint32_t ef = b.top() >> 23;  // exponent field; 0 (zero, subnormal) clamps like 1 does
  uint32_t scale = ef > 2u ? ef - 2u : 0u;
  uint32_t code[4] = {0u, 0u, 0u, 0u};
  if (ef == 255u) {
    scale = 255u;
  } else {
    const float inv = __uint_as_float((254u - scale) << 23);  // 2^(127 - scale), normal
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[8];
      b.eight(j, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= inv;
      code[j] = e2m1x8(v);
    }
  }
  reinterpret_cast<uint4*>(a.codes)[u] = make_uint4(code[0], code[1], code[2], code[3]);
  unsigned char* s = a.scales + row * a.scols + c;
  *s = static_cast<unsigned char>(scale);
  if (c + 1u == a.bpr)  // the row's last block also clears the padding bytes
    for (unsigned p = c + 1u; p < a.scols; ++p) *++s = 0;
}

template <class Out>
__global__ void __launch_bounds__(kMxThreads) mrs_mxfp4_dequantize_kernel(const MxDequantArgs a) {
  pdl_trigger();
  const size_t u = static_cast<size_t>(blockIdx.x) * kMxThreads + threadIdx.x;
  const size_t row = u / a.bpr;
  const unsigned c = static_cast<unsigned>(u - row * a.bpr);
  pdl_wait();
  if (u >= a.blocks) return;
  const uint4 q = __ldg(reinterpret_cast<const uint4*>(a.codes) + u);
  const float s = e8m0_value(__ldg(a.scales + row * a.scols + c));
  const uint32_t code[4] = {q.x, q.y, q.z, q.w};
  Out* y = static_cast<Out*>(a.y) + row * a.stride + 32 * static_cast<size_t>(c);
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v[8];
    e2m1_values(code[j], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s;
    if constexpr (sizeof(Out) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
      store32(y + 8 * j, a.wide != 0, w);
    } else {
      // the one rounding of this direction: exact in bf16 down to its smallest subnormal
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[4 * (j & 1) + i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if (j & 1) store32(y + 8 * (j - 1), a.wide != 0, w);
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
  // (the launch has a CTA per 256 blocks of 32)
  if (rows > (int64_t{1} << 40) || stride > (int64_t{1} << 40) ||
      rows * (cols / 32) > int64_t{INT32_MAX} * kMxThreads / 4)
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
  a.bpr = static_cast<unsigned>(cols / 32);
  a.blocks = static_cast<size_t>(rows) * a.bpr;
  a.stride = static_cast<size_t>(x_stride);
  a.wide = aligned(x, 32) && static_cast<size_t>(x_stride) * size % 32 == 0;
  a.scols = static_cast<unsigned>(scols);
  a.codes = codes;
  a.scales = scales;
  const dim3 grid(static_cast<unsigned>((a.blocks + kMxThreads - 1) / kMxThreads));
  auto* k = x_dtype == MOE_RS_FP32   ? mrs_mxfp4_quantize_kernel<BlockFp32>
            : x_dtype == MOE_RS_FP16 ? mrs_mxfp4_quantize_kernel<BlockHalf<false>>
                                     : mrs_mxfp4_quantize_kernel<BlockHalf<true>>;
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
  a.bpr = static_cast<unsigned>(cols / 32);
  a.blocks = static_cast<size_t>(rows) * a.bpr;
  a.stride = static_cast<size_t>(y_stride);
  a.wide = aligned(y, 32) && static_cast<size_t>(y_stride) * size % 32 == 0;
  a.scols = static_cast<unsigned>(scols);
  a.y = y;
  const dim3 grid(static_cast<unsigned>((a.blocks + kMxThreads - 1) / kMxThreads));
  auto* k = y_dtype == MOE_RS_FP32 ? mrs_mxfp4_dequantize_kernel<float>
                                   : mrs_mxfp4_dequantize_kernel<__nv_bfloat16>;
  return launch_status(launch_pdl(k, grid, dim3(kMxThreads), 0, stream, a));
}

}  // extern "C"
