// mrs_product_grad.cu -- gradient of the experts' products' weights.
//
// For every expert e, m < outs, k < cols:
//   grad_w[e, m, k] = sum over routes r of e in the list of G[row, m] * X[row', k]
// with fp32 sums, rounded once.  The contraction runs over the ragged rows of an expert, which lie
// one behind another in the sorted list: both operands are copied row by row, so that in shared
// memory each position of the contraction is a line of consecutive m (or k), the transposed layout
// of the tensor core.  Rows past an expert's last are zeros.
//
// A pair of CTAs computes tiles of 256 m by 256 k of one expert, 64 rows a step; each CTA brings
// 128 m and 128 k.  The tasks of the warps are those of mrs_product.cu.  Experts without routes get
// their zeros from the storing warps alone.  Two sets of eight warps copy the steps in turn, so that
// one set's look at the list is hidden behind the other's copies; tiles leave by tensor copies.
//
// T = 8192, E = 64, topk = 8, 2048 x 7168: 1570 to 1700 us, of 996 at the tensor cores' rate.  Bound
// by the copies: both operands are rows somewhere in memory, a thread's copy takes 16 bytes, and an SM
// takes in 512 bytes of such copies every 16 clocks, the 32 KB of a step in 1024 clocks or so where
// its products need 512.  T = 1000, E = 129, 264 x 520: 24.9 us, the storing warps' latency for ten tiles
// of one step each.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mrs_product.cuh"

namespace mrs {

struct WeightGradArgs {
  ListArgs list;
  int32_t* status;
  const unsigned char *g, *x;
  unsigned long long wait_limit_ns;
  int topk, g_per_route, x_per_route;
  int E, N, K;
  int mtiles, ktiles;
  int type, out_type;
};

constexpr int kGradCopiers = 8;          // warps that copy a step, four for each operand
constexpr int kGradTurns = 2;            // steps go to so many sets of them in turn
constexpr int kGradThreads = 32 * (12 + kGradTurns * kGradCopiers);
constexpr int kGradTmem = 512;
// (Five slots and a second stage for each storing warp: T = 8192, E = 64, 2048 x 7168 1600 us and 1570 so,
// E = 128, 768 x 3584 408 and 378; T = 1000, E = 129, 264 x 520 24.5 and 24.9.)
constexpr int kGradSlots = 6;
constexpr int kGradInfo = 16;  // units ahead: where they have one step each, all slots are on their way
constexpr int kGradUsers = 9 + kGradTurns * kGradCopiers;  // eight storing warps, copies, their announcer
constexpr int kGradDeep = 64;            // rows of a step
// Steps from which a tile's sums are made in two accumulators, half of the rows each: the tensor core
// cuts where an addition would round, and sums come out low by 1e-9 of themselves for every row, 1e-6
// over 1024.  fp32 results that have more rows give up the overlap of the next tile's products with the
// stores (T = 8192, E = 64, 2048 x 7168: 1570 us with a limit of 1024 rows, 1690 with 512, 1550 with
// 4096); in 16 bits it does not show before 4096 rows.
template <class Out>
constexpr int kGradLong = sizeof(Out) == 4 ? 16 : 64;
constexpr int kGradTile = 128 * 128;     // bytes of an operand in a CTA and step
constexpr int kGradStage = 32 * 128;     // of a storing warp: 128 bytes of 32 rows
constexpr size_t kGradSmem =
    static_cast<size_t>(kGradSlots) * 2 * kGradTile + 8 * kGradStage + 1024;

// Waits that last as long as a tile takes (its storing warps', and the list's for a unit to be done)
// have the limit once more for every 2^21 rows: 33 M clocks of products and copies, 6 % of the default
// limit.  (With one limit whatever the rows, experts of 25 million rows and more gave up.)
__device__ __forceinline__ unsigned long long grad_limit(unsigned long long limit, unsigned rows) {
  return limit * (1u + (rows >> 21));
}

struct GradInfo {
  int e, p0, rows, m0, k0;  // e < 0: no more units
};
__device__ __forceinline__ int grad_steps(unsigned rows) { return (rows + kGradDeep - 1) / kGradDeep; }

template <class Out>
__global__ void __launch_bounds__(kGradThreads, 1)
    mrs_weight_grad_kernel(const __grid_constant__ CUtensorMap omap, const WeightGradArgs a) {
  constexpr int S = kGradSlots;
  extern __shared__ unsigned char smem_raw[];
  __shared__ unsigned long long rows_s[S], free_s[S], full_s[S], acc_full_s[2], acc_free_s[2],
      info_full_s[kGradInfo], info_free_s[kGradInfo], done_s;
  __shared__ GradInfo info_s[kGradInfo];
  __shared__ uint32_t tmem_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(pair_rank());
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t gbase = base, xbase = base + S * kGradTile;
  const unsigned long long limit = a.wait_limit_ns;
  pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&rows_s[s], 32 * kGradCopiers);
      mbar_init(&free_s[s], 1);
      mbar_init(&full_s[s], 2);  // both CTAs' rows
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full_s[b], 1);
      mbar_init(&acc_free_s[b], 16);
    }
    for (int i = 0; i < kGradInfo; ++i) {
      mbar_init(&info_full_s[i], 1);
      mbar_init(&info_free_s[i], kGradUsers + (rank == 0 ? 1 : 0));  // and the products
    }
    mbar_init(&done_s, 1);
    fence_mbar_init();
  }
  if (warp == 2) pair_tmem_alloc(&tmem_s, kGradTmem);
  tc_fence_before();
  __syncthreads();
  pair_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  pdl_wait();

  bool ok = true;
  Ring<kGradInfo> at_info;
  auto next_unit = [&]() -> const GradInfo* {
    ok = ok && warp_wait(&info_full_s[at_info.slot], at_info.phase, limit);
    if (!ok) return nullptr;
    const GradInfo* q = &info_s[at_info.slot];
    return q->e < 0 ? nullptr : q;
  };
  auto leave_unit = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&info_free_s[at_info.slot]);
    at_info.advance();
  };

  if (warp >= 12) {
    // a warp copies 16 rows of a step of one operand, 256 bytes of two rows at a time
    Ring<S> at;
    const bool is_x = ((warp - 12) & 4) != 0;
    const int turn = (warp - 12) / kGradCopiers;
    int now = 0;  // whose step it is
    const int w16 = 16 * (warp & 3), chunk = lane & 15, sub = lane >> 4;
    const int per_route = is_x ? a.x_per_route : a.g_per_route, cols = is_x ? a.K : a.N;
    const unsigned char* from = is_x ? a.x : a.g;
    const size_t row_bytes = 2 * static_cast<size_t>(cols);
    const uint32_t place = (is_x ? xbase : gbase) + (chunk >> 3) * (kGradDeep * 128) +
                           (w16 + sub) * 128;
    while (const GradInfo* q = next_unit()) {
      // (what looks past the last row is counted without a sign: a list has up to 2^31 - 1 rows)
      const int p0 = q->p0;
      const unsigned rows = q->rows;
      const int col = (is_x ? q->k0 : q->m0) + 128 * rank + 8 * chunk;
      const bool in = col < cols;
      const unsigned char* mine = from + (in ? 2 * static_cast<size_t>(col) : 0);
      // lanes 0 to 15 look up a row each, four steps ahead (one step ahead every step took as long as
      // the access: 2200 us for T = 8192, E = 64, 7168 -> 2048)
      auto route_of = [&](unsigned first) {
        const unsigned r = first + w16 + lane;
        return lane < 16 && r < rows ? __ldg(a.list.sid + p0 + r) : -1;
      };
      int ahead[4];
      const int skipped = (turn - now + kGradTurns) % kGradTurns, steps = grad_steps(rows);
      constexpr unsigned kStride = kGradTurns * kGradDeep;
      const unsigned r1 = skipped * kGradDeep;
      at.skip(min(skipped, steps));
#pragma unroll
      for (int k = 0; k < 4; ++k) ahead[k] = route_of(r1 + k * kStride);
      for (unsigned r4 = r1; r4 < rows; r4 += 4 * kStride) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const unsigned r0 = r4 + k * kStride;
          if (r0 >= rows) break;
          const int r = ahead[k] >= 0 && ahead[k] < a.list.routes
                            ? (per_route ? ahead[k] : ahead[k] / a.topk) : -1;
          ahead[k] = route_of(r0 + 4 * kStride);
          int row[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) row[j] = __shfl_sync(kFull, r, 2 * j + sub);
          ok = ok && thread_wait(&free_s[at.slot], at.phase ^ 1u, limit);
          if (ok) {  // (a lane whose wait gave up goes along until the unit ends)
            if (r0 + w16 < rows) {  // (no product takes rows behind the last 16 that hold one)
              const uint32_t to = place + at.slot * kGradTile;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const bool is = row[j] >= 0;
                // (columns behind the last meet no output)
                if (in)
                  copy16(to + 256 * j + 16 * ((chunk & 7) ^ ((2 * j + sub) & 7)),
                         mine + (is ? row[j] * row_bytes : 0), is ? 16 : 0);
              }
            }
            copy_arrive(&rows_s[at.slot]);
          }
          at.skip(min(kGradTurns, steps - static_cast<int>(r0 / kGradDeep)));
        }
      }
      now = (now + steps) % kGradTurns;
      ok = __all_sync(kFull, ok);
      leave_unit();
    }
    copy_wait_all();
  } else if (warp == 1) {
    const int each = a.mtiles * a.ktiles, units = a.E * each, step = gridDim.x >> 1;
    const ListArgs& l = a.list;
    // the owners (most of them, for long lists) come while the list's length does
    int touched = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int b = 1024 * k + 32 * lane;
      if (b < l.max_rows >> l.log2B)
        asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(touched) : "l"(l.eid + b));
    }
    const int blocks = min(max(__ldg(l.npp), 0), l.max_rows) >> l.log2B;
    unsigned most = 0;  // rows of a unit so far
    for (int u0 = blockIdx.x >> 1; ok && u0 < units; u0 += 32 * step) {
      // a lane looks up one of the next 32 units: the run of its expert's blocks, and the rows of it
      // up to the last route (routes come first in its last block)
      const long long u = u0 + static_cast<long long>(lane) * step;
      int e = -1, p0 = 0, rows = 0, m0 = 0, k0 = 0;
      if (u < units) {
        e = static_cast<int>(u) / each;
        const int i = static_cast<int>(u) - e * each, mt = i / a.ktiles;
        m0 = mt * 256;
        k0 = (i - mt * a.ktiles) * 256;
        int b0, b1;
        prefix_lengths(blocks, [&](int b) { return __ldg(l.eid + b); }, e, b0, b1);
        const int n = max(b1 - b0, 0);
        p0 = b0 * l.B;
        if (n > 0) {
          const int32_t* last = l.sid + p0 + (n - 1) * l.B;
          rows = (n - 1) * l.B + prefix_length(l.B, [&](int i) {
                   const int r = __ldg(last + i);
                   return r >= 0 && r < l.routes;
                 });
        }
      }
      for (int i = 0; ok && i < 32; ++i) {
        const int ei = __shfl_sync(kFull, e, i);
        if (ei < 0) break;
        ok = warp_wait(&info_free_s[at_info.slot], at_info.phase ^ 1u, grad_limit(limit, most));
        if (!ok) break;
        most = max(most, static_cast<unsigned>(__shfl_sync(kFull, rows, i)));
        if (lane == i) {
          info_s[at_info.slot] = GradInfo{e, p0, rows, m0, k0};
          mbar_arrive(&info_full_s[at_info.slot]);
        }
        __syncwarp();
        at_info.advance();
      }
    }
    ok = ok && warp_wait(&info_free_s[at_info.slot], at_info.phase ^ 1u, grad_limit(limit, most));
    if (ok && lane == 0) {
      info_s[at_info.slot].e = -1;
      mbar_arrive(&info_full_s[at_info.slot]);
    }
    // the searches take owners in order: every CTA looks at some
    bool bad = false;
    for (unsigned b = blockIdx.x * 32 + lane; b < static_cast<unsigned>(blocks); b += gridDim.x * 32) {
      const int e = __ldg(l.eid + b);
      bad |= e < 0 || e >= a.E || (b > 0 && __ldg(l.eid + b - 1) > e);
    }
    if (bad) atomicOr(a.status, MOE_RS_DEVICE_BAD_EXPERT_ID);
  } else if (warp == 3) {
    // announces the rows that threads have written to the tensor cores
    Ring<S> at;
    while (const GradInfo* q = next_unit()) {
      const int steps = grad_steps(q->rows);
      if (elect_one()) {
        Ring<S> s = at;
        for (int i = 0; ok && i < steps; ++i) {
          ok = thread_wait(&rows_s[s.slot], s.phase, limit);
          if (!ok) break;
          fence_proxy_async_smem();
          pair_arrive_first(&full_s[s.slot]);
          s.advance();
        }
      }
      ok = __all_sync(kFull, ok);
      at.skip(steps);
      leave_unit();
    }
  } else if (warp == 2 && rank == 0) {
    Ring<S> at;
    int buf = 0;
    uint32_t acc_phase = 0;
    bool any = false;
    const uint32_t word = pair_word(a.type, true, true, 256);
    while (const GradInfo* q = next_unit()) {
      const unsigned rows = q->rows;
      const int steps = grad_steps(rows);
      if (steps > 0) {
        any = true;
        if (elect_one()) {
          Ring<S> s = at;
          int into = buf;
          const int second = steps > kGradLong<Out> ? steps / 2 : steps;  // its first step
          ok = pair_wait(&acc_free_s[buf], acc_phase ^ 1u, limit);
          for (int ks = 0; ok && ks < steps; ++ks) {
            if (ks == second) {
              pair_commit(&acc_full_s[into]);
              into ^= 1;
              ok = pair_wait(&acc_free_s[into], acc_phase ^ (buf == 0 ? 1u : 0u), limit);
              if (!ok) break;
            }
            ok = pair_wait(&full_s[s.slot], s.phase, limit);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dg = desc_lines128(gbase + s.slot * kGradTile, kGradDeep);
            const uint64_t dx = desc_lines128(xbase + s.slot * kGradTile, kGradDeep);
            const int parts = (min(rows - ks * kGradDeep, 64u) + 15) >> 4;
#pragma unroll
            for (int g = 0; g < 4; ++g)
              if (g < parts)  // else rows past the last: zeros
                pair_mma<false>(tmem + into * 256, dg + 128 * g, dx + 128 * g, word,
                                (ks > 0 && ks != second) || g > 0);
            pair_commit(&free_s[s.slot]);
            s.advance();
          }
          if (ok) pair_commit(&acc_full_s[into]);
        }
        ok = __all_sync(kFull, ok);
        at.skip(steps);
        if (steps > kGradLong<Out>) {  // both, and back to this one
          acc_phase ^= 1u;
        } else if (++buf == 2) {
          buf = 0;
          acc_phase ^= 1u;
        }
      }
      leave_unit();
    }
    if (any) {
      if (elect_one()) pair_commit_first(&done_s);
      __syncwarp();
      warp_wait(&done_s, 0, kWaitLimitNs);
    }
  } else if (warp >= 4 && warp < 12) {
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t stage = base + S * 2 * kGradTile + (warp - 4) * kGradStage;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    int buf = 0;
    uint32_t acc_phase = 0;
    while (const GradInfo* q = next_unit()) {
      const int m = q->m0 + 128 * rank + 32 * quarter, k0 = q->k0, e = q->e;
      const bool some = q->rows > 0, both = q->rows > kGradLong<Out> * kGradDeep;
      if (some) {
        const unsigned long long whole = grad_limit(limit, q->rows);
        ok = warp_wait(&acc_full_s[buf], acc_phase, whole);
        if (!ok) break;
        if (both) {
          ok = warp_wait(&acc_full_s[buf ^ 1], acc_phase ^ (buf == 0 ? 0u : 1u), whole);
          if (!ok) break;
        }
        tc_fence_after();
      }
      const uint32_t src = tmem + buf * 256 + lanes, src2 = tmem + (buf ^ 1) * 256 + lanes;
      // Tiles of 32 rows by 128 bytes go through shared memory, in the swizzle of the tensor copy that
      // stores them.  (Lanes that store 32 bytes of a row each take 32 lines an access, beside the
      // copies that wait for the same unit.)
      constexpr int kCols = 128 / sizeof(Out);
      const int last = m < a.N ? min(256, a.K - k0) : 0;
#pragma unroll 1
      for (int c0 = kCols * half; c0 < last; c0 += 2 * kCols) {
        uint32_t w[32];  // the lane's row of the tile
#pragma unroll
        for (int part = 0; part < kCols / 32; ++part) {
          uint32_t v[32];
          __syncwarp();
          if (some) {
            tmem_load32(src + c0 + 32 * part, v);
            tmem_wait(v);
            if (both) {
#pragma unroll
              for (int c = 0; c < 32; c += 8) tmem_add8(src2 + c0 + 32 * part + c, v + c);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = 0u;
          }
          if constexpr (sizeof(Out) == 4) {
#pragma unroll
            for (int c = 0; c < 32; ++c) w[c] = v[c];
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float lo = __uint_as_float(v[2 * c]), hi = __uint_as_float(v[2 * c + 1]);
              if (a.out_type == MOE_RS_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
                w[16 * part + c] = *reinterpret_cast<const uint32_t*>(&h);
              } else {
                const __half2 h = __floats2half2_rn(lo, hi);
                w[16 * part + c] = *reinterpret_cast<const uint32_t*>(&h);
              }
            }
          }
        }
        if (lane == 0) tma_store_read();  // what was there has been read
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                           stage + 128 * lane + 16 * (c ^ (lane & 7))),
                       "r"(w[4 * c]), "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                       : "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tma_store_3d(&omap, stage, k0 + c0, m, e);
      }
      if (some) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) pair_arrive_first(&acc_free_s[buf]);
        if (both) {
          if (lane == 0) pair_arrive_first(&acc_free_s[buf ^ 1]);
          acc_phase ^= 1u;
        } else if (++buf == 2) {
          buf = 0;
          acc_phase ^= 1u;
        }
      }
      leave_unit();
    }
    if (lane == 0) tma_store_done();  // (a CTA that leaves takes its shared memory along)
    __syncwarp();
  }
  if (!ok && lane == 0) atomicOr(a.status, MOE_RS_DEVICE_WAIT_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  pair_sync();
  tc_fence_after();
  if (warp == 2) pair_tmem_free(tmem, kGradTmem);
}

namespace {

template <class Out>
cudaError_t launch_weight_grad(const CUtensorMap& o, const WeightGradArgs& a, int pairs,
                               cudaStream_t st) {
  auto* k = mrs_weight_grad_kernel<Out>;
  static SmemGrant granted;
  const cudaError_t err = grant_smem(reinterpret_cast<const void*>(k), kGradSmem, granted);
  if (err != cudaSuccess) return err;
  return launch_pairs(k, pairs, kGradThreads, kGradSmem, st, o, a);
}

}  // namespace
}  // namespace mrs

using namespace mrs;

extern "C" int moe_experts_grad_weights(
    const void* grad, int dtype, int g_per_route, const void* x, int x_per_route, int T, int E,
    int topk, int cols, int outs, int block_m, const int32_t* sorted_token_ids,
    const int32_t* expert_ids, const int32_t* num_tokens_post_pad, void* grad_w, int out_dtype,
    void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (T < 0) return MOE_RS_ERR_BAD_TOKENS;
  if (E < 1 || E > kMaxExperts) return MOE_RS_ERR_BAD_EXPERTS;
  if (topk < 1 || topk > kMaxTopk) return MOE_RS_ERR_BAD_TOPK;
  if (block_m < 1 || block_m > 1024 || (block_m & (block_m - 1)) != 0)
    return MOE_RS_ERR_BAD_BLOCK_M;
  if (dtype != MOE_RS_BF16 && dtype != MOE_RS_FP16) return MOE_RS_ERR_BAD_DTYPE;
  if (out_dtype != dtype && out_dtype != MOE_RS_FP32) return MOE_RS_ERR_BAD_DTYPE;
  if (cols < 8 || cols > MOE_RS_PRODUCT_MAX_COLS || cols % 8 != 0 || outs < 8 ||
      outs > MOE_RS_PRODUCT_MAX_COLS || outs % 8 != 0)
    return MOE_RS_ERR_BAD_COLS;
  if (static_cast<int64_t>(T) * topk > INT32_MAX ||
      static_cast<int64_t>(moe_sort_max_padded(T, E, topk, block_m)) > INT32_MAX)
    return MOE_RS_ERR_OVERFLOW;
  const size_t need = moe_experts_product_workspace_bytes(T, E, topk, block_m);
  if (!workspace || workspace_bytes < need) return MOE_RS_ERR_WORKSPACE;
  const size_t routes = static_cast<size_t>(T) * topk;
  const size_t out_size = out_dtype == MOE_RS_FP32 ? 4 : 2;
  const size_t n = static_cast<size_t>(E) * outs * cols;
  if (!grad_w) return MOE_RS_ERR_NULL_POINTER;
  if (T > 0 && (!grad || !x || !sorted_token_ids || !expert_ids || !num_tokens_post_pad))
    return MOE_RS_ERR_NULL_POINTER;
  if (!aligned(grad, 16) || !aligned(x, 16) || !aligned(sorted_token_ids, 4) ||
      !aligned(expert_ids, 4) || !aligned(num_tokens_post_pad, 4) || !aligned(grad_w, 16) ||
      !aligned(workspace, 16))
    return MOE_RS_ERR_MISALIGNED;
  if (T == 0)  // no route of any expert
    return launch_status(cudaMemsetAsync(grad_w, 0, n * out_size, stream));
  const size_t grows = g_per_route ? routes : static_cast<size_t>(T);
  const size_t xrows = x_per_route ? routes : static_cast<size_t>(T);
  const size_t P = moe_sort_max_padded(T, E, topk, block_m);
  const Span outs_s[] = {span(grad_w, n * out_size), span(workspace, workspace_bytes)};
  const Span ins[] = {span(grad, 2 * grows * outs), span(x, 2 * xrows * cols),
                      span(sorted_token_ids, 4 * P), span(expert_ids, 4 * (P / block_m)),
                      span(num_tokens_post_pad, 4)};
  if (any_alias(outs_s, 2, ins, 5)) return MOE_RS_ERR_ALIAS;
  const int64_t units = static_cast<int64_t>(E) * ((outs + 255) / 256) * ((cols + 255) / 256);
  if (units > INT32_MAX / 2) return MOE_RS_ERR_OVERFLOW;
  const int sms = sm_count();
  if (sms == 0) return launch_status(cudaErrorInvalidDevice);
  WeightGradArgs a{};
  a.list.eid = expert_ids;
  a.list.sid = sorted_token_ids;
  a.list.npp = num_tokens_post_pad;
  a.list.E = E;
  a.list.B = block_m;
  while ((1 << a.list.log2B) < block_m) ++a.list.log2B;
  a.list.max_rows = static_cast<int>(P);
  a.status = static_cast<int32_t*>(workspace);
  a.g = static_cast<const unsigned char*>(grad);
  a.x = static_cast<const unsigned char*>(x);
  a.wait_limit_ns = product_wait_limit();
  a.list.routes = static_cast<int>(routes);
  a.topk = topk;
  a.g_per_route = g_per_route != 0;
  a.x_per_route = x_per_route != 0;
  a.E = E;
  a.N = outs;
  a.K = cols;
  a.mtiles = (outs + 255) / 256;
  a.ktiles = (cols + 255) / 256;
  a.type = dtype == MOE_RS_BF16 ? 1 : 0;
  a.out_type = out_dtype;
  CUtensorMap map;
  if (!encode_weights3(&map, grad_w, out_dtype, static_cast<int>(out_size), cols, outs, E, 32))
    return MOE_RS_ERR_LAUNCH;
  const int pairs = units < sms / 2 ? static_cast<int>(units) : sms / 2;
  return launch_status(out_dtype == MOE_RS_FP32
                           ? launch_weight_grad<float>(map, a, pairs, stream)
                           : launch_weight_grad<uint16_t>(map, a, pairs, stream));
}
