// mrs_product.cuh -- what the experts' products in 16 and 8 bits and their gradients share: how a
// call's sorted list is searched and cut into row tiles, and the host side of tensor maps.
#pragma once

#include <climits>
#include <cstdint>

#include "mrs_args.h"
#include "mrs_internal.h"
#include "mrs_tc.cuh"

namespace mrs {

// The workspace: the status word, the number of tiles, and the tiles of lists that are too long for a
// CTA to cut by itself.
struct ProductTable {
  int32_t* head;   // [0] status bits (sticky), [1] tiles
  int4* tiles;     // expert, first row of the list, rows, -
};
constexpr int kTileRowsLeast = 64;

inline size_t product_table_bytes(size_t max_tiles) { return 256 + sizeof(int4) * max_tiles; }
inline ProductTable product_table(void* workspace) {
  char* p = static_cast<char*>(workspace);
  return ProductTable{reinterpret_cast<int32_t*>(p), reinterpret_cast<int4*>(p + 256)};
}

// Of n places whose first ones satisfy `is`, how many do: quarters are looked at side by side, so that
// it takes half as many accesses one behind another as halves.  (Where others do too the answer is some
// number up to n.)
template <class P>
__device__ __forceinline__ int prefix_length(int n, P&& is) {
  int lo = 0;
  while (n > 0) {
    const int q = (n + 3) >> 2;
    int c = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) c += is(lo + min((i + 1) * q, n) - 1) ? 1 : 0;
    const int before = min(c * q, n), last = min(before + q, n);
    lo += before;
    n = c == 3 ? n - before : last - before - 1;  // (the last of the quarter does not)
  }
  return lo;
}

// How many of n ascending values are below v, and how many are not above it: two such searches at
// once, which take no longer than one.  (Of values in another order: some numbers up to n.)
template <class V>
__device__ __forceinline__ void prefix_lengths(int n, V&& value, int v, int& below, int& upto) {
  // (without a sign: four quarters of 2^31 - 1 values end past them)
  unsigned lo[2] = {0, 0}, m[2] = {static_cast<unsigned>(n), static_cast<unsigned>(n)};
  while (m[0] > 0 || m[1] > 0) {
    int x[2][3];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 3; ++i)
        x[k][i] = m[k] > 0 ? value(lo[k] + min((i + 1u) * ((m[k] + 3) >> 2), m[k]) - 1) : 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (m[k] == 0) continue;
      const unsigned q = (m[k] + 3) >> 2;
      unsigned c = 0;
#pragma unroll
      for (int i = 0; i < 3; ++i) c += x[k][i] < v + k ? 1 : 0;
      const unsigned before = min(c * q, m[k]), last = min(before + q, m[k]);
      lo[k] += before;
      // (of values in another order nothing may be left before the last)
      m[k] = c == 3 ? m[k] - before : (last > before ? last - before - 1 : 0);
    }
  }
  below = lo[0];
  upto = lo[1];
}

// The sorted list of a call.
struct ListArgs {
  const int32_t *eid, *sid, *npp;
  int E, B, log2B, max_rows, routes;
  int rows, log2R;  // rows of a tile at most
  int by_used;    // tiles of a run alike, up to its last route; else of `rows` each, up to its last block
};

// The product of a few routes, straight from the list; its weights' map.
bool encode_few(CUtensorMap* map, const void* p, size_t row_bytes, size_t rows, size_t E);
struct FewArgs {
  const unsigned char* x;
  const int32_t *sid, *eid, *npp;
  const float *sw, *xs, *ws;  // or null
  int32_t* status;
  void* out;
  unsigned long long wait_limit_ns;
  int routes, topk, per_route, E, N, K, B, blocks, out_type;
  int nchunk, ksteps;  // set by the launch
};
cudaError_t launch_product_few(const CUtensorMap& wmap, FewArgs a, int type, int sms,
                               cudaStream_t st);

// E matrices of `size`-byte elements; a box is 128 bytes of `box_rows` rows of one, swizzled by 128.
// What lies outside reads as zero and is not stored.
bool encode_weights3(CUtensorMap* map, const void* p, int type, int size, size_t cols, size_t rows,
                     size_t E, int box_rows);

// Waits give up after the test hook's limit, but not before whatever a CTA has in flight has had
// ample time to land.
inline unsigned long long product_wait_limit() {
  const unsigned long long v = debug_wait_limit_ns();
  return v == 0ull || v > 5000000ull ? v : 5000000ull;
}

// Launch in clusters of two CTAs, ordered like launch_pdl.
template <class... Params, class... Args>
cudaError_t launch_pairs(void (*kernel)(Params...), int pairs, int threads, size_t smem,
                         cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// A place in a ring of S slots, and the parity of its round.
template <int S>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance() {
    if (++slot == S) {
      slot = 0;
      phase ^= 1u;
    }
  }
  __device__ __forceinline__ void skip(int steps) {
    const int to = slot + steps;
    phase ^= static_cast<uint32_t>(to / S) & 1u;
    slot = to % S;
  }
};

}  // namespace mrs
