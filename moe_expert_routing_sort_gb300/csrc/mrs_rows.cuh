// mrs_rows.cuh -- what the operators on rows share (norm, gated activation, rows to 8 bits): how
// a row is laid over threads, 16-byte vectors of its elements, reductions over a row, e4m3 codes.
//
// A row of `cols` elements (a multiple of 8) is cols / 8 vectors.  `tpr` threads take a row, kVec
// vectors each, vector i of a thread being number i * tpr + (its place): neighbours read side by
// side.  Rows of up to 128 vectors are taken by 8, 16 or 32 lanes and reduced by shuffles; wider
// ones by whole warps, which meet in shared memory.  A CTA has several short rows.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "mrs_args.h"
#include "mrs_internal.h"

namespace mrs {

constexpr int kRowMaxCols = MOE_RS_ROWS_MAX_COLS;  // 2 vectors a thread, 1024 threads
// Three or four vectors a thread are those of rows within a warp, whose CTAs are small.
template <int kVec>
constexpr int kRowThreads = kVec > 2 ? 256 : 1024;

// ------------------------------------------------------------------------------ vectors
template <class T>
__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
// One rounding, to nearest even.
template <class T>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <class T>
__device__ __forceinline__ uint4 load8(const void* base, size_t element) {
  return __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(base) + element));
}
// Elements 8 i .. 8 i + 7 of a vector over columns, of the rows' type or fp32.
template <class T>
__device__ __forceinline__ void load_columns(const void* p, bool f32, int i, float (&v)[8]) {
  if (f32) {
    const float4 a = __ldg(static_cast<const float4*>(p) + 2 * i);
    const float4 b = __ldg(static_cast<const float4*>(p) + 2 * i + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    unpack8<T>(load8<T>(p, 8 * static_cast<size_t>(i)), v);
  }
}

// --------------------------------------------------------------------------- 8-bit rows
// A row's scale is its largest magnitude / 448 (the largest e4m3 value), at least 2^-126 so that
// its reciprocal is finite; a row that holds an infinity or a NaN takes a NaN for its scale and
// codes of zero, so that it reads back as NaN.  `top`: the largest magnitude's bits (ordered like
// the magnitudes, infinities and NaN on top).
__device__ __forceinline__ float fp8_scale(uint32_t top) {
  if (top >= 0x7f800000u) return __uint_as_float(0x7fffffffu);
  return fmaxf(__uint_as_float(top) / 448.0f, __uint_as_float(0x00800000u));
}
// What a value is multiplied by ahead of its rounding; 0 of a row that reads back as NaN.  The
// product is one rounding of 2^-24 away from the quotient, ahead of one of 2^-4.
__device__ __forceinline__ float fp8_inverse(float scale) {
  return scale == scale ? 1.0f / scale : 0.0f;
}
// Eight values to codes, to nearest even, saturating at 448.
__device__ __forceinline__ uint2 fp8_codes(const float (&v)[8], float inv) {
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // (inv is 0 where a value may be an infinity or a NaN)
    const float lo = inv == 0.0f ? 0.0f : v[2 * i] * inv, hi = inv == 0.0f ? 0.0f : v[2 * i + 1] * inv;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(hi), "f"(lo));
  }
  return make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16),
                    h[2] | (static_cast<uint32_t>(h[3]) << 16));
}
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// ---------------------------------------------------------------------------- reductions
// Sum and largest bits over a row's threads, in an order fixed by the shape; every thread gets
// both.  meet: shared memory of the CTA, a float and a word for each warp.  Every thread of the
// CTA calls it where rows are wider than a warp.
struct RowTotals {
  float sum;
  uint32_t top;
};
__device__ __forceinline__ RowTotals row_totals(float sum, uint32_t top, int tpr, RowTotals* meet) {
  const int lanes = tpr < 32 ? tpr : 32;
  for (int o = lanes >> 1; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(kFull, sum, o);
    top = max(top, __shfl_xor_sync(kFull, top, o));
  }
  if (tpr <= 32) return RowTotals{sum, top};
  const int warps = tpr >> 5, warp = static_cast<int>(threadIdx.x) >> 5;
  const int first = warp / warps * warps;
  if ((threadIdx.x & 31) == 0) meet[warp] = RowTotals{sum, top};
  __syncthreads();
  RowTotals r{0.0f, 0u};
  for (int w = 0; w < warps; ++w) {
    const RowTotals q = meet[first + w];
    r.sum += q.sum;
    r.top = max(r.top, q.top);
  }
  __syncthreads();  // the next row's totals may be written
  return r;
}

// ---------------------------------------------------------------------------- host side
struct RowPlan {
  int vec;      // vectors of a thread: 1 to 4
  int tpr;      // threads of a row
  int rows;     // rows of a CTA
  int threads;
};
// `most`: vectors that a thread takes at most where the row allows it.
inline RowPlan row_plan(int cols, int most, int threads = 256) {
  const int v = cols / 8;
  RowPlan p{};
  if (v <= 8) {
    p.tpr = 8;
  } else if (v <= 128) {  // the lanes that leave the fewest idle; the most of those that tie
    p.tpr = 32;
    for (int lanes = 16; lanes >= 8; lanes >>= 1)
      if ((v + lanes - 1) / lanes <= 4 &&
          (v + lanes - 1) / lanes * lanes < (v + p.tpr - 1) / p.tpr * p.tpr)
        p.tpr = lanes;
  } else {
    const int vec = v <= 1024 * most ? most : 2;
    p.tpr = ((v + vec - 1) / vec + 31) / 32 * 32;
  }
  p.vec = (v + p.tpr - 1) / p.tpr;
  p.rows = p.tpr >= threads ? 1 : threads / p.tpr;
  p.threads = p.rows * p.tpr;
  return p;
}

// Rows of `cols` elements of `size` bytes, `stride` elements apart, as a span.
inline Span rows_span(const void* p, int64_t rows, int64_t cols, int64_t stride, size_t size) {
  return span(p, p == nullptr || rows == 0
                     ? 0
                     : (static_cast<size_t>(rows - 1) * static_cast<size_t>(stride) +
                        static_cast<size_t>(cols)) * size);
}

}  // namespace mrs
