// mrs_packed.cu -- the operations of training, rows and experts behind one call that takes its arguments
// as an array: for bindings that pay for every argument they convert (20 arguments through ctypes
// take 1.8 us on the host, an array of them 0.5, and a small call's kernel 4).
#include <climits>
#include <cstdint>
#include <cstring>
#include <tuple>
#include <type_traits>

#include "moe_route_sort.h"

namespace {

// Arguments in turn.  A number outside its type's range marks the whole call.
struct Packed {
  const int64_t* at;
  bool fits = true;
  int64_t next() { return *at++; }
  template <class T>
  T* ptr() {
    return reinterpret_cast<T*>(static_cast<uintptr_t>(next()));
  }
  int num() {
    const int64_t v = next();
    if (v < INT_MIN || v > INT_MAX) fits = false;
    return static_cast<int>(v);
  }
  size_t size() {
    const int64_t v = next();
    if (v < 0) fits = false;
    return static_cast<size_t>(v);
  }
  float real() {
    double d;
    const int64_t v = next();
    std::memcpy(&d, &v, sizeof d);
    return static_cast<float>(d);
  }
  cudaStream_t stream() { return ptr<CUstream_st>(); }
  template <class A>
  A get() {
    if constexpr (std::is_pointer_v<A>) return ptr<std::remove_pointer_t<A>>();
    else if constexpr (std::is_same_v<A, float>) return real();
    else if constexpr (std::is_same_v<A, int>) return num();
    else if constexpr (std::is_same_v<A, size_t>) return size();
    else return next();
  }
};

// `fn` with the n arguments that follow, each as fn's declaration has it.
template <class... A>
int call(int (*fn)(A...), int64_t n, Packed& p) {
  if (n != static_cast<int64_t>(sizeof...(A))) return MOE_RS_ERR_BAD_CALL;
  const std::tuple<A...> args{p.get<A>()...};  // (braces: from the first to the last)
  if (!p.fits) return MOE_RS_ERR_OVERFLOW;
  return std::apply(fn, args);
}

}  // namespace

extern "C" int moe_call_packed(const void* args) {
  if (!args) return MOE_RS_ERR_NULL_POINTER;
  if (reinterpret_cast<uintptr_t>(args) % 8 != 0) return MOE_RS_ERR_MISALIGNED;
  Packed p{static_cast<const int64_t*>(args)};
  const int64_t op = p.next(), n = p.next();
  switch (op) {
    case MOE_RS_CALL_BALANCE_LOSS: {
      if (n != 15) return MOE_RS_ERR_BAD_CALL;
      const void* x = p.ptr<const void>();
      const int32_t* ids = p.ptr<const int32_t>();
      const int32_t* off = p.ptr<const int32_t>();
      const int T = p.num(), E = p.num(), K = p.num(), S = p.num(), softmax = p.num();
      const float coef = p.real();
      float* loss = p.ptr<float>();
      int32_t* counts = p.ptr<int32_t>();
      float* mean = p.ptr<float>();
      void* ws = p.ptr<void>();
      const size_t bytes = p.size();
      cudaStream_t st = p.stream();
      if (!p.fits) return MOE_RS_ERR_OVERFLOW;
      return moe_balance_loss(x, ids, off, T, E, K, S, softmax, coef, loss, counts, mean, ws,
                              bytes, st);
    }
    case MOE_RS_CALL_ROUTE_BACKWARD: {
      if (n != 16) return MOE_RS_ERR_BAD_CALL;
      const void* x = p.ptr<const void>();
      const int32_t* ids = p.ptr<const int32_t>();
      const float* gw = p.ptr<const float>();
      const float* gl = p.ptr<const float>();
      const int32_t* counts = p.ptr<const int32_t>();
      const int32_t* off = p.ptr<const int32_t>();
      const int T = p.num(), E = p.num(), K = p.num(), S = p.num(), softmax = p.num();
      const float R = p.real(), coef = p.real();
      void* out = p.ptr<void>();
      const int dtype = p.num();
      cudaStream_t st = p.stream();
      if (!p.fits) return MOE_RS_ERR_OVERFLOW;
      return moe_route_backward(x, ids, gw, gl, counts, off, T, E, K, S, softmax, R, coef, out,
                                dtype, st);
    }
    case MOE_RS_CALL_MXFP4_QUANTIZE: {
      if (n != 8) return MOE_RS_ERR_BAD_CALL;
      const void* x = p.ptr<const void>();
      const int dtype = p.num();
      const int64_t rows = p.next();
      const int cols = p.num();
      const int64_t stride = p.next();
      uint8_t* codes = p.ptr<uint8_t>();
      uint8_t* scales = p.ptr<uint8_t>();
      cudaStream_t st = p.stream();
      if (!p.fits) return MOE_RS_ERR_OVERFLOW;
      return moe_mxfp4_quantize(x, dtype, rows, cols, stride, codes, scales, st);
    }
    case MOE_RS_CALL_MXFP4_DEQUANTIZE: {
      if (n != 8) return MOE_RS_ERR_BAD_CALL;
      const uint8_t* codes = p.ptr<const uint8_t>();
      const uint8_t* scales = p.ptr<const uint8_t>();
      const int64_t rows = p.next();
      const int cols = p.num();
      void* y = p.ptr<void>();
      const int dtype = p.num();
      const int64_t stride = p.next();
      cudaStream_t st = p.stream();
      if (!p.fits) return MOE_RS_ERR_OVERFLOW;
      return moe_mxfp4_dequantize(codes, scales, rows, cols, y, dtype, stride, st);
    }
    case MOE_RS_CALL_EXPERTS_MXFP4: {
      if (n != 20) return MOE_RS_ERR_BAD_CALL;
      const uint8_t* xc = p.ptr<const uint8_t>();
      const uint8_t* xs = p.ptr<const uint8_t>();
      const int per_route = p.num();
      const uint8_t* wc = p.ptr<const uint8_t>();
      const uint8_t* ws = p.ptr<const uint8_t>();
      const int T = p.num(), E = p.num(), K = p.num(), cols = p.num(), outs = p.num();
      const int block_m = p.num();
      const int32_t* sid = p.ptr<const int32_t>();
      const float* sw = p.ptr<const float>();
      const int32_t* eid = p.ptr<const int32_t>();
      const int32_t* npp = p.ptr<const int32_t>();
      void* out = p.ptr<void>();
      const int dtype = p.num();
      void* work = p.ptr<void>();
      const size_t bytes = p.size();
      cudaStream_t st = p.stream();
      if (!p.fits) return MOE_RS_ERR_OVERFLOW;
      return moe_experts_mxfp4(xc, xs, per_route, wc, ws, T, E, K, cols, outs, block_m, sid, sw,
                               eid, npp, out, dtype, work, bytes, st);
    }
    case MOE_RS_CALL_FP8_QUANTIZE: return call(moe_fp8_quantize, n, p);
    case MOE_RS_CALL_RMS_NORM: return call(moe_rms_norm, n, p);
    case MOE_RS_CALL_RMS_NORM_BACKWARD: return call(moe_rms_norm_backward, n, p);
    case MOE_RS_CALL_SWIGLU: return call(moe_swiglu, n, p);
    case MOE_RS_CALL_SWIGLU_BACKWARD: return call(moe_swiglu_backward, n, p);
    case MOE_RS_CALL_EXPERTS_PRODUCT: return call(moe_experts_product, n, p);
    case MOE_RS_CALL_EXPERTS_GRAD_ROWS: return call(moe_experts_grad_rows, n, p);
    case MOE_RS_CALL_EXPERTS_GRAD_WEIGHTS: return call(moe_experts_grad_weights, n, p);
    default: return MOE_RS_ERR_BAD_CALL;
  }
}
