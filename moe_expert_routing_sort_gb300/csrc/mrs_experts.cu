// mrs_experts.cu -- the experts' products of MXFP4 rows and weights, driven by the sort step.
//
// For every row p of the sorted list that is a route r = sorted_token_ids[p] (r < T * topk), with
// e the owner of its block:
//   out[r, n] = w_p * sum over k of X[row(r), k] W[e, n, k],   row(r) = r, or r / topk
// X and W are E2M1 codes with one E8M0 scale per 32 columns; sums are fp32, the row's weight
// (1 without weights) is applied in fp32, and the result is rounded once to the output type.
//
// One tile is the rows of one block (the M side of the tensor-core product, 128 lanes of tensor
// memory; blocks of more rows are cut, blocks of fewer leave lanes unused) by 128 outputs of its
// expert (the N side).  Rows on the lanes make the result a row per thread, so the outputs leave
// as 32-byte stores of whole sectors; a block of 16 rows costs the tensor core as much as one of
// 128, which it has time for: such calls wait for the weights.  A persistent CTA per SM takes
// tiles round robin, the output tiles of a block next to each other, so the SMs share a block's
// rows and an expert's weights in L2.  Steps of 256 columns (128 bytes a row) go through a ring of
// shared-memory stages; the warps of a CTA each have one task:
//   0      copies the weights' 128 rows (a tensor copy, in the 128-byte swizzle that
//          the tensor core reads)
//   1      copies the step's scales to tensor memory and issues four products of 64
//          columns; the tensor core applies the scales and adds into fp32 in tensor memory
//   4-7    a finished tile from tensor memory to the output rows, while the next one is computed
//          (two accumulators)
//   8-11   the block's rows, 16 bytes a thread into the same swizzle; the copies arrive on the
//          stage's barrier themselves, so the whole ring is in flight.  (Gathered by tensor copies
//          of four rows each they took 37 ns a copy: 1.2 us a step of 128 rows, against 0.14 us
//          of products.)
//   12-15  the scales of rows and weights, from row-major bytes to the order that tensor memory
//          wants (row r of 128: lane r % 32, word r / 32 of 4 scales)
// Each task has the list entries of the next two tiles and the first scales of the next one in
// flight, so a tile of two steps does not wait for them.  Every wait is bounded; a wait that gives
// up ends its warp's task with the status bit set, and the CTA leaves once nothing of its own is
// in flight.
#include <cuda_bf16.h>

#include "mrs_args.h"
#include "mrs_internal.h"
#include "mrs_tc.cuh"

namespace mrs {

struct ExpertsArgs {
  const unsigned char *xc, *xs, *ws;  // rows, their scales, the weights' scales
  const int32_t* sid;
  const float* sw;  // or null
  const int32_t* eid;
  const int32_t* npp;
  int32_t* status;
  void* out;
  unsigned long long wait_limit_ns;
  int routes, topk, per_route;
  int E, K, N, B, scols, max_rows;
  int sub, subs;   // rows of a tile (<= 128), tiles along a block's rows
  int ntile;       // tiles along the outputs
  int ksteps;      // steps of 256 columns
  int wide_scales; // scale rows start on 16 bytes
  int wide_out;    // output rows start on 32 bytes
};

constexpr int kExpThreads = 512;  // warps 2 and 3 only fill the quarter of the epilogue's lanes
constexpr int kExpRows = 128;      // lanes of a tile: rows of a block
constexpr int kExpOuts = 128;      // outputs of a tile
constexpr int kStepBytes = 128;    // bytes of a row per step
constexpr int kXBytes = kExpRows * kStepBytes;
constexpr int kWBytes = kExpOuts * kStepBytes;
constexpr int kScaleBytes = 2048;  // rows' and weights' scales of a step: 2 x 2 x 512
constexpr int kStageBytes = kXBytes + kWBytes + kScaleBytes;
constexpr int kStages = 6;         // what fits in 227 KB
constexpr size_t kExpSmem = static_cast<size_t>(kStages) * kStageBytes + 1024;
constexpr int kTmemCols = 512;     // 2 accumulators of 128 columns, 16 of scales per stage
constexpr int kTmemScales = 2 * kExpOuts;

// A tile of the list: its expert id is in flight or here (-1 past the last tile).
struct ExpertsTile {
  int it, p0, n0, e;
  __device__ __forceinline__ void at(const ExpertsArgs& a, int i, int tiles) {
    it = i;
    const int b = i / a.ntile;
    n0 = (i - b * a.ntile) * kExpOuts;
    p0 = b * a.sub;
    e = i < tiles ? __ldg(a.eid + b / a.subs) : -1;
  }
  __device__ __forceinline__ bool valid(const ExpertsArgs& a) const { return e >= 0 && e < a.E; }
  // Entry i of the tile's rows (-1: a lane unused, or past the last tile).
  __device__ __forceinline__ int entry(const ExpertsArgs& a, int i, int tiles) const {
    return (it < tiles && i < a.sub) ? __ldg(a.sid + p0 + i) : -1;
  }
};

// Scales of one row, 16 bytes (two steps) at a time; zeros past the row's end and for null rows.
// Nothing here looks at what it loads: a use would wait for it.
__device__ __forceinline__ uint4 load_scales(const unsigned char* row, int pair, const ExpertsArgs& a) {
  const int at = 16 * pair, left = a.K / 32 - at;
  uint4 q = make_uint4(0u, 0u, 0u, 0u);
  if (row == nullptr || left <= 0) return q;
  if (a.wide_scales) return __ldg(reinterpret_cast<const uint4*>(row + at));
  const uint32_t* p = reinterpret_cast<const uint32_t*>(row + at);
  q.x = __ldg(p);
  if (left > 4) q.y = __ldg(p + 1);
  if (left > 8) q.z = __ldg(p + 2);
  if (left > 12) q.w = __ldg(p + 3);
  return q;
}

// The first `left` bytes of four scales: what lies behind a row's K / 32 scales is padding, and
// its columns' products of zeros have to meet a finite scale.
__device__ __forceinline__ uint32_t keep_scales(uint32_t w, int left) {
  return left >= 4 ? w : (left <= 0 ? 0u : w & ((1u << (8 * left)) - 1u));
}

__device__ __forceinline__ void store_shared(uint32_t dst, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst), "r"(v) : "memory");
}

// Where the scales of row r of 128 start in a step's 512 bytes.
__device__ __forceinline__ uint32_t scale_place(int r) { return 16 * (r & 31) + 4 * (r >> 5); }

template <class Out>
__global__ void __launch_bounds__(kExpThreads, 1)
    mrs_experts_kernel(const __grid_constant__ CUtensorMap wmap, const ExpertsArgs a) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ unsigned long long full_s[kStages], empty_s[kStages], acc_full_s[2], acc_free_s[2],
      done_s;
  __shared__ uint32_t tmem_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const unsigned long long limit = a.wait_limit_ns;
  pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      // the weights' copy, the scales' four warps, the threads of the warps that copy rows
      mbar_init(&full_s[s], 1 + 4 + 32 * ((a.sub + 31) / 32));
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
  const int tiles = rows / a.B * a.subs * a.ntile;
  const int step = gridDim.x;
  bool ok = true;
  int stage = 0;
  uint32_t phase = 0;  // parity of the ring's current round
  auto advance = [&] {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  };
  ExpertsTile t, n;
  t.at(a, blockIdx.x, tiles);

  if (warp == 0) {
    long long issued = 0;
    for (; ok && t.it < tiles; t = n) {
      n.at(a, t.it + step, tiles);
      if (!t.valid(a)) {
        if (lane == 0) atomicOr(a.status, MOE_RS_DEVICE_BAD_EXPERT_ID);
        continue;
      }
      for (int ks = 0; ks < a.ksteps; ++ks) {
        ok = warp_wait(&empty_s[stage], phase ^ 1u, limit);
        if (!ok) break;
        if (elect_one()) {
          mbar_expect(&full_s[stage], kWBytes);
          tma_load_3d(base + stage * kStageBytes + kXBytes, &wmap, ks * kStepBytes, t.n0, t.e,
                      &full_s[stage]);
        }
        __syncwarp();
        ++issued;
        advance();
      }
    }
    if (!ok) {
      // a copy still on its way must land before the CTA leaves; the phase it completes may be
      // missing other arrivals, so this waits for what has no one to take it any more
      for (long long q = issued > kStages ? issued - kStages : 0; q < issued; ++q)
        warp_wait(&full_s[q % kStages], static_cast<uint32_t>(q / kStages) & 1u, kWaitLimitNs);
    }
  } else if (warp == 1) {
    int buf = 0;
    uint32_t acc_phase = 0;
    bool any = false;
    for (; ok && t.it < tiles; t = n) {
      n.at(a, t.it + step, tiles);
      if (!t.valid(a)) continue;
      ok = warp_wait(&acc_free_s[buf], acc_phase ^ 1u, limit);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + buf * kExpOuts;
      for (int ks = 0; ks < a.ksteps; ++ks) {
        ok = warp_wait(&full_s[stage], phase, limit);
        if (!ok) break;
        tc_fence_after();
        fence_proxy_async_smem();  // the rows were written by threads
        const uint32_t src = base + stage * kStageBytes, sc = src + kXBytes + kWBytes;
        const uint32_t ts = tmem + kTmemScales + stage * 16;
        const uint64_t dx = desc_rows128(src), dw = desc_rows128(src + kXBytes);
        const int parts = (a.K - 256 * ks + 63) >> 6;
        if (elect_one()) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            tc_copy_scales(ts + 4 * g, desc_scales(sc + 512 * g));
            tc_copy_scales(ts + 8 + 4 * g, desc_scales(sc + 1024 + 512 * g));
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < parts)  // else columns past K
              // 32 bytes further along the swizzled rows: 2 units of 16
              tc_mma_mxf4(d, dx + 2 * q, dw + 2 * q, mxf4_word(kExpRows, kExpOuts, (q & 1) * 2),
                          ts + 4 * (q >> 1), ts + 8 + 4 * (q >> 1), ks > 0 || q > 0);
          tc_commit(&empty_s[stage]);
          if (ks + 1 == a.ksteps) tc_commit(&acc_full_s[buf]);
        }
        __syncwarp();
        any = true;
        advance();
      }
      buf ^= 1;
      if (buf == 0) acc_phase ^= 1u;
    }
    // nothing of the tensor core may be in flight when tensor memory is given back
    if (any) {
      if (elect_one()) tc_commit(&done_s);
      __syncwarp();
      warp_wait(&done_s, 0, kWaitLimitNs);
    }
  } else if (warp >= 4 && warp < 8) {
    const int i = 32 * (warp - 4) + lane;  // the thread's row of a tile
    const bool used = 32 * (warp - 4) < a.sub;
    int buf = 0;
    uint32_t acc_phase = 0;
    int entry = t.entry(a, i, tiles);
    for (; ok && t.it < tiles; t = n) {
      n.at(a, t.it + step, tiles);
      const int r = entry;
      entry = n.entry(a, i, tiles);
      if (!t.valid(a)) continue;
      const bool put = r >= 0 && r < a.routes;
      const float w = (a.sw != nullptr && put) ? __ldg(a.sw + t.p0 + i) : 1.0f;
      ok = warp_wait(&acc_full_s[buf], acc_phase, limit);
      if (!ok) break;
      if (used) {
        tc_fence_after();
        const uint32_t src = tmem + buf * kExpOuts + (static_cast<uint32_t>(32 * (warp - 4)) << 16);
        Out* out = static_cast<Out*>(a.out) + (put ? static_cast<size_t>(r) * a.N : 0) + t.n0;
        const int left = a.N - t.n0;  // a multiple of 8
#pragma unroll
        for (int c0 = 0; c0 < kExpOuts; c0 += 32) {
          uint32_t v[32];
          tmem_load32(src + c0, v);
          if constexpr (sizeof(Out) == 4) {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(w * __uint_as_float(v[c]));
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(w * __uint_as_float(v[2 * c]),
                                                             w * __uint_as_float(v[2 * c + 1]));
              v[c] = *reinterpret_cast<const uint32_t*>(&h);
            }
          }
          constexpr int kPer = 32 / sizeof(Out);  // outputs of 32 bytes
#pragma unroll
          for (int c = 0; put && c < 32 / kPer; ++c) {
            const int at = c0 + kPer * c;
            const uint32_t* q = v + 8 * c;
            void* o = out + at;
            if (a.wide_out && at + kPer <= left) {
              asm volatile(
                  "st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "r"(q[0]),
                  "r"(q[1]), "r"(q[2]), "r"(q[3]), "r"(q[4]), "r"(q[5]), "r"(q[6]), "r"(q[7])
                  : "memory");
            } else {
              uint4* o4 = static_cast<uint4*>(o);
              if (at + kPer / 2 <= left) o4[0] = make_uint4(q[0], q[1], q[2], q[3]);
              if (at + kPer <= left) o4[1] = make_uint4(q[4], q[5], q[6], q[7]);
            }
          }
          __syncwarp();
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_free_s[buf]);
      buf ^= 1;
      if (buf == 0) acc_phase ^= 1u;
    }
  } else if (warp >= 8 && warp < 12) {
    // warp w copies rows 32 w .. 32 w + 31 of the block, four rows (8 lanes each) at a time
    const int w32 = 32 * (warp - 8);
    const int mine = min(a.sub - w32, 32);  // rows of this warp
    const int chunk = lane & 7, sub4 = lane >> 3;
    const size_t half = static_cast<size_t>(a.K / 2);
    // row 4 j + sub4 of the warp: two swizzles, for even and odd j
    const uint32_t place = (w32 + sub4) * kStepBytes;
    const uint32_t even = place + 16 * (chunk ^ sub4), odd = place + 16 * (chunk ^ (sub4 + 4));
    if (mine > 0) {
      int entry = t.entry(a, w32 + lane, tiles);
      for (; ok && t.it < tiles; t = n) {
        n.at(a, t.it + step, tiles);
        const int r = entry;
        entry = n.entry(a, w32 + lane, tiles);
        if (!t.valid(a)) continue;
        const int src = r >= 0 && r < a.routes ? (a.per_route ? r : r / a.topk) : -1;
        // rows that are no route keep what was there: any codes, in rows that are not stored
        const unsigned char* from[8];
        unsigned has = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int s = __shfl_sync(kFull, src, 4 * j + sub4);
          from[j] = a.xc + static_cast<size_t>(max(s, 0)) * half + 16 * chunk;
          has |= s >= 0 ? 1u << j : 0u;
        }
        for (int ks = 0; ks < a.ksteps; ++ks) {
          ok = warp_wait(&empty_s[stage], phase ^ 1u, limit);
          if (!ok) break;
          const uint32_t dst = base + stage * kStageBytes;
          // (columns past K keep what was there too: they meet weights that read as zero)
          const unsigned live = ks * kStepBytes + 16 * chunk < a.K / 2 ? has : 0u;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (4 * j >= mine) break;
            if ((live >> j) & 1u) copy16(dst + ((j & 1) ? odd : even) + 512 * j, from[j]);
            from[j] += kStepBytes;
          }
          copy_arrive(&full_s[stage]);
          advance();
        }
      }
      copy_wait_all();
    }
  } else if (warp >= 12) {
    // a thread has one row of the block and one of the weights
    const int i = tid - 384;
    ExpertsTile f;
    n.at(a, t.it + step, tiles);
    auto xrow = [&](const ExpertsTile& q, int r) -> const unsigned char* {
      if (!q.valid(a) || r < 0 || r >= a.routes) return nullptr;
      return a.xs + static_cast<size_t>(a.per_route ? r : r / a.topk) * a.scols;
    };
    auto wrow = [&](const ExpertsTile& q) -> const unsigned char* {
      return q.valid(a) && q.n0 + i < a.N
                 ? a.ws + (static_cast<size_t>(q.e) * a.N + q.n0 + i) * a.scols
                 : nullptr;
    };
    const unsigned char *px = xrow(t, t.entry(a, i, tiles)), *pw = wrow(t);
    int entry = n.entry(a, i, tiles);
    uint4 firstx = load_scales(px, 0, a), firstw = load_scales(pw, 0, a);
    const uint32_t place = base + kXBytes + kWBytes + scale_place(i);
    for (; ok && t.it < tiles; t = n, n = f) {
      f.at(a, n.it + step, tiles);
      const unsigned char *nx = xrow(n, entry), *nw = wrow(n);
      entry = f.entry(a, i, tiles);
      uint4 cx, cw, ax = firstx, aw = firstw;
      uint4 bx = load_scales(px, 1, a), bw = load_scales(pw, 1, a);
      firstx = load_scales(nx, 0, a);
      firstw = load_scales(nw, 0, a);
      if (t.valid(a)) {
        for (int ks = 0; ks < a.ksteps; ++ks) {
          if ((ks & 1) == 0) {
            cx = ax;
            cw = aw;
            ax = bx;
            aw = bw;
            bx = load_scales(px, ks / 2 + 2, a);
            bw = load_scales(pw, ks / 2 + 2, a);
          } else {
            cx.x = cx.z;
            cx.y = cx.w;
            cw.x = cw.z;
            cw.y = cw.w;
          }
          ok = warp_wait(&empty_s[stage], phase ^ 1u, limit);
          if (!ok) break;
          const uint32_t dst = place + stage * kStageBytes;
          const int left = a.K / 32 - 8 * ks;
          if (left < 8) {
            cx.x = keep_scales(cx.x, left);
            cx.y = keep_scales(cx.y, left - 4);
            cw.x = keep_scales(cw.x, left);
            cw.y = keep_scales(cw.y, left - 4);
          }
          store_shared(dst, cx.x);
          store_shared(dst + 512, cx.y);
          store_shared(dst + 1024, cw.x);
          store_shared(dst + 1536, cw.y);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full_s[stage]);
          advance();
        }
      }
      px = nx;
      pw = nw;
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

// The weights: `outs` rows of `row` bytes for each of E experts; the copied box is 128 bytes of
// 128 rows of one expert (rows past the last and bytes past the row's end read as zero).
bool encode_weights(CUtensorMap* map, const void* p, size_t row, size_t outs, size_t E) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {row, outs, E};
  const cuuint64_t strides[2] = {row, row * outs};
  const cuuint32_t box[3] = {kStepBytes, kExpOuts, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(p), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Out>
cudaError_t launch_experts(const CUtensorMap& wmap, const ExpertsArgs& a, int grid,
                           cudaStream_t st) {
  auto* k = mrs_experts_kernel<Out>;
  static SmemGrant granted;
  const cudaError_t err = grant_smem(reinterpret_cast<const void*>(k), kExpSmem, granted);
  if (err != cudaSuccess) return err;
  return launch_pdl(k, dim3(grid), dim3(kExpThreads), kExpSmem, st, wmap, a);
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
  const bool f32 = out_dtype == MOE_RS_FP32;
  const int64_t tiles = static_cast<int64_t>(P / block_m) *
                        ((block_m + kExpRows - 1) / kExpRows) *
                        ((outs + kExpOuts - 1) / kExpOuts);
  if (tiles > INT32_MAX / 2) return MOE_RS_ERR_OVERFLOW;
  const int sms = sm_count();
  if (sms == 0) return launch_status(cudaErrorInvalidDevice);
  ExpertsArgs a{};
  a.xc = x_codes;
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
  a.sub = block_m < kExpRows ? block_m : kExpRows;
  a.subs = block_m / a.sub;
  a.ntile = (outs + kExpOuts - 1) / kExpOuts;
  a.ksteps = (cols + 255) / 256;
  a.wide_scales = scols % 16 == 0 && aligned(x_scales, 16) && aligned(w_scales, 16);
  a.wide_out = aligned(out, 32) && outs * (f32 ? 4 : 2) % 32 == 0;
  CUtensorMap wmap;
  if (!encode_weights(&wmap, w_codes, cols / 2, outs, E)) return MOE_RS_ERR_LAUNCH;
  const int grid = tiles < sms ? static_cast<int>(tiles) : sms;
  return launch_status(f32 ? launch_experts<float>(wmap, a, grid, stream)
                           : launch_experts<__nv_bfloat16>(wmap, a, grid, stream));
}

}  // extern "C"
