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

// Two fp32 values side by side, one instruction for both.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2_pair(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float f2_sum(F2 a) {
  const float2 p = f2_pair(a);
  return p.x + p.y;
}
template <class T>
__device__ __forceinline__ void unpack8(const uint4& q, F2 (&v)[4]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[i] = f2(f.x, f.y);
    }
  }
}
template <class T>
__device__ __forceinline__ uint4 pack8(const F2 (&v)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = f2_pair(v[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
  return pack8<T>(f);
}
template <class T>
__device__ __forceinline__ void load_columns(const void* p, bool f32, int i, F2 (&v)[4]) {
  float f[8];
  load_columns<T>(p, f32, i, f);
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = f2(f[2 * k], f[2 * k + 1]);
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
// Eight values times `inv` (1 / scale) to codes, to nearest even, saturating at 448.  The product is
// two roundings of 2^-24 away from the quotient, ahead of one of 2^-4.
__device__ __forceinline__ uint2 fp8_codes(const float (&v)[8], float inv) {
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(h[i])
        : "f"(v[2 * i + 1] * inv), "f"(v[2 * i] * inv));
  return make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16),
                    h[2] | (static_cast<uint32_t>(h[3]) << 16));
}
// A row's codes where its scale is a number, zeros otherwise.
__device__ __forceinline__ uint2 fp8_codes_of(const float (&v)[8], float scale) {
  return scale == scale ? fp8_codes(v, 1.0f / scale) : make_uint2(0u, 0u);
}
__device__ __forceinline__ uint2 fp8_codes_of(const F2 (&v)[4], float scale) {
  if (scale != scale) return make_uint2(0u, 0u);
  const float inv = 1.0f / scale;
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = f2_pair(v[i] * f2(inv, inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(p.y), "f"(p.x));
  }
  return make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16),
                    h[2] | (static_cast<uint32_t>(h[3]) << 16));
}
// The larger magnitude, a NaN where one is.
__device__ __forceinline__ float larger(float top, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(top), "f"(fabsf(v)));
  return r;
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
  if (tpr < 32) {
    for (int o = tpr >> 1; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(kFull, sum, o);
      top = max(top, __shfl_xor_sync(kFull, top, o));
    }
    return RowTotals{sum, top};
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  top = __reduce_max_sync(kFull, top);
  if (tpr == 32) return RowTotals{sum, top};
  const int warps = tpr >> 5, warp = static_cast<int>(threadIdx.x) >> 5, lane = threadIdx.x & 31;
  const int first = warp / warps * warps;
  if (lane == 0) meet[warp] = RowTotals{sum, top};
  __syncthreads();
  RowTotals r{0.0f, 0u};
  if (lane < warps) r = meet[first + lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r.sum += __shfl_xor_sync(kFull, r.sum, o);
  r.top = __reduce_max_sync(kFull, r.top);
  __syncthreads();  // the next row's totals may be written
  return r;
}

// ------------------------------------------------------------------------ rows in flight
// A stream of 16-byte vectors from global memory through shared memory, kDepth items of kVec vectors
// ahead.  A thread copies and reads its own vectors alone, so that nothing has to be met: each item is
// one group of background copies, and the oldest group has landed once kDepth - 1 are left.  (Loads
// into registers wait for a row's reduction before the next row's are on their way: 59 us for 8192
// rows of 3584, 318 for the gradient of 8192 rows of 7168 with eight rows a token.)
template <int kVec, int kDepth>
struct RowStream {
  static_assert((kDepth & (kDepth - 1)) == 0, "");
  uint32_t mine, slot_bytes, to = 0, from = 0;  // this thread's first vector; places in the ring
  uint32_t off[kVec];                           // of this thread's vectors in a row
  int count = 0;                                // that it has
  __device__ __forceinline__ RowStream(void* smem, int place, int tpr, int vecs)
      : mine(static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + 16 * threadIdx.x),
        slot_bytes(16 * kVec * blockDim.x) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      off[i] = 16u * (i * tpr + place);
      count += i * tpr + place < vecs ? 1 : 0;
    }
  }
  // The next item, a row that starts at `row`, if there is one.
  __device__ __forceinline__ void put(bool is, const unsigned char* row) {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (is && i < count)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine + to +
                                                                       16 * i * blockDim.x),
                     "l"(row + off[i])
                     : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
    to += slot_bytes;
    if (to == kDepth * slot_bytes) to = 0;
  }
  // The oldest item.
  __device__ __forceinline__ void get(uint4 (&v)[kVec]) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                   : "r"(mine + from + 16 * i * blockDim.x)
                   : "memory");
    from += slot_bytes;
    if (from == kDepth * slot_bytes) from = 0;
  }
  static __host__ __device__ size_t bytes(int threads) { return static_cast<size_t>(16) * kVec * kDepth * threads; }
};
// Items ahead: 128 bytes a thread, 256 where a CTA has an SM to itself.
template <int kVec>
constexpr int kRowDepth = kVec == 1 ? 8 : (kVec == 2 ? 4 : 2);

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

// CTAs that the device holds at once, as far as threads (of 64 registers) and shared memory go.
inline int64_t row_ctas(int threads, size_t smem, int sms) {
  const int by_threads = 1024 / threads, by_smem = static_cast<int>((224 * 1024) / (smem + 1536));
  const int n = by_threads < by_smem ? by_threads : by_smem;
  return static_cast<int64_t>(sms) * (n < 1 ? 1 : n);
}

// Rows of `cols` elements of `size` bytes, `stride` elements apart, as a span.
inline Span rows_span(const void* p, int64_t rows, int64_t cols, int64_t stride, size_t size) {
  return span(p, p == nullptr || rows == 0
                     ? 0
                     : (static_cast<size_t>(rows - 1) * static_cast<size_t>(stride) +
                        static_cast<size_t>(cols)) * size);
}

}  // namespace mrs
